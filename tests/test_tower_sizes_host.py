"""What the tower operators' size queries promise over whole ranges of sizes (CPU: the queries are
host-pure, no compute call is made here)."""
import random

import pytest

from embedding_lookup_feature_amd import tower as tw

MIB = 1 << 20


def test_group_norm_forward_workspace_is_bounded():
    """At most 8 MiB for up to 2048 channels, whatever the batch and the positions."""
    r = random.Random(7)
    shapes = [(1492, 9, 1888, 32), (1182, 11, 1696, 32), (704, 10, 1824, 32)]
    for _ in range(60_000):
        C = max(1, round(2 ** r.uniform(0, 11)))
        G = r.choice([g for g in (1, 2, 3, 4, 8, 16, 32, C) if C % g == 0])
        shapes.append((round(2 ** r.uniform(0, 18)), round(2 ** r.uniform(0, 14)), C, G))
    for s in shapes:
        assert tw.group_norm_fwd_workspace_bytes(*s) <= 8 * MIB, s


def test_workspaces_of_the_measured_range_fit_a_programs_buffers():
    """The buffers that perf/operators.py gives its calls hold for every size that it draws."""
    op = pytest.importorskip("perf.operators")
    give = {"group_norm_fwd": 8 * MIB, "group_norm_train": 64 * MIB, "dense_fwd": 160 * MIB, "dense_bwd": 512 * MIB}
    r = random.Random(11)
    for _ in range(60_000):
        c = op.draw(r)
        if c["op"].startswith("group_norm"):
            a = (c["M"], c["S"], c["C"], c["G"])
            need = tw.group_norm_fwd_workspace_bytes(*a)
            if c["op"] == "group_norm_train":
                need = max(need, tw.group_norm_bwd_workspace_bytes(*a))
        elif c["op"].startswith("dense"):
            a = (c["M"], c["K"], c["N"])
            need = (tw.dense_fwd_workspace_bytes if c["op"] == "dense_fwd" else tw.dense_bwd_workspace_bytes)(*a)
        else:
            continue
        assert need <= give[c["op"]], (c["op"], a, need)


A = 0x7F0000000000  # fake, aligned: every call below ends at its checks


@pytest.mark.parametrize("M,N,extra", [(1 << 29, 8, 1), (2**31 - 1, 8, 0), (1 << 29, 1, 8), (1 << 24, 1 << 13, 1)])
def test_dense_outputs_of_too_many_tiles_are_refused_before_any_work(M, N, extra):
    """Also where operands would be copied first (odd row strides): nothing is enqueued, so the
    refusal is the call's and no launch is tried."""
    from embedding_lookup_feature_amd import embcore as ec
    L, K, big = tw.lib(), 8, 1 << 50
    rc = L.el_dense_fwd(A, K + extra, M, K, A, None, N, 0, None, None, 0, None, 0, A, N, ec.EL_BF16, A, big, None)
    assert rc == ec.EL_ERR_UNSUPPORTED and "tiles" in ec.el_last_error()
    assert tw.dense_fwd_workspace_bytes(M, K, N) == 0
    # the data gradient's output is [M, K]: the sizes the other way round
    rc = L.el_dense_bwd(A, N + extra, M, N, A, K, A, K + extra, None, 0, A, N, 0, None, None, 0, None, 0, A, None,
                        ec.EL_BF16, A, big, None)
    assert rc == ec.EL_ERR_UNSUPPORTED and "tiles" in ec.el_last_error()


def test_dense_sizes_up_to_the_limit_pass_the_checks():
    """One tile below the limit the call goes on to ask for its workspace."""
    from embedding_lookup_feature_amd import embcore as ec
    M, K, N = (1 << 29) - 256, 8, 8
    rc = tw.lib().el_dense_fwd(A, K + 1, M, K, A, None, N, 0, None, None, 0, None, 0, A, N, ec.EL_BF16, None, 0, None)
    assert rc == ec.EL_ERR_WORKSPACE
    assert tw.dense_fwd_workspace_bytes(M, K, N) >= 16 * M


def test_dense_bwd_partials_are_counted_for_the_longest_batches():
    r256, pad8 = (lambda n: -(-n // 256) * 256), (lambda n: -(-n // 8) * 8)
    for M in (2**31 - 1, 2**31 - 64, 2**31 - 65, 2**31 - 4096):
        for K, N in ((8, 1 << 20), (1 << 20, 8), (8, 8), (512, 1024)):
            copies = sum(r256(a * pad8(b) * 2) for a, b in ((M, N), (M, K), (N, K)))
            assert tw.dense_bwd_workspace_bytes(M, K, N) - copies >= 4 * N * K, (M, K, N)


def test_group_norm_takes_every_pooled_vector_of_the_largest_batch_as_a_row():
    """26 tables x 262144 samples of 128 channels as rows (one position each), and as many as one
    launch's grid of several samples per workgroup holds."""
    from embedding_lookup_feature_amd import embcore as ec
    L, big = tw.lib(), 1 << 50
    fwd = lambda B, S, C, G, ws=A, n=big: L.el_group_norm_fwd(  # noqa: E731
        A, C, B, S, C, G, None, None, None, -1.0, 0, A, C, A, A, ec.EL_BF16, ws, n, None)
    bwd = lambda B, S, C, G, ws, n: L.el_group_norm_bwd(  # noqa: E731
        A, C, A, C, B, S, C, G, None, None, None, A, A, 0, A, C, A, A, ec.EL_BF16, ws, n, None)
    for B, C, G in ((26 * 262144, 128, 1), ((1 << 25) - 1, 64, 1), ((1 << 24), 512, 1), ((1 << 22) + 1, 4096, 1)):
        assert fwd(B, 1, C, G) == ec.EL_ERR_INVALID_ARG and "eps" in ec.el_last_error(), (B, C, G)  # past the sizes
        assert bwd(B, 1, C, G, None, 0) == ec.EL_ERR_WORKSPACE
        assert tw.group_norm_bwd_workspace_bytes(B, 1, C, G) > 0
    for B, S, C, G in ((1 << 25, 1, 64, 1), ((1 << 23) + 1, 1, 4096, 1), ((1 << 22), 1, 64, 8), ((1 << 22) + 1, 4096, 64, 1)):
        assert fwd(B, S, C, G) == ec.EL_ERR_UNSUPPORTED, (B, S, C, G)
        assert bwd(B, S, C, G, A, big) == ec.EL_ERR_UNSUPPORTED
        assert tw.group_norm_bwd_workspace_bytes(B, S, C, G) == 0 == tw.group_norm_fwd_workspace_bytes(B, S, C, G)


def test_binding_refuses_sizes_beyond_32_bits(monkeypatch):
    """A row count that a 32-bit argument would cut (2^32 + 4 rows to 4) is refused by the binding,
    not handed on; samples times positions may pass 2^31."""
    import torch
    calls = []

    class FakeLibrary:
        def __getattr__(self, name):
            return (lambda *a: 4096) if name.endswith("workspace_bytes") else (lambda *a: calls.append((name, a)) or 0)

    monkeypatch.setattr(tw, "lib", FakeLibrary)
    monkeypatch.setattr(tw, "_mat", lambda t, name, shape, dtype: (A, shape[1]))
    monkeypatch.setattr(tw, "_vec", lambda *a: A)
    monkeypatch.setattr(tw, "_stream", lambda *a: 0)
    monkeypatch.setattr(tw.ec, "_dev", lambda t, name: A)
    m = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    ws = torch.empty(4096, dtype=torch.uint8)
    many, few = 2**32 + 4, 16
    for bad in (
            lambda: tw.act_dropout_fwd(m(many, 1), m(many, 1)),
            lambda: tw.act_dropout_fwd(m(1, many), m(1, many)),
            lambda: tw.act_dropout_bwd(m(many, 1), None, m(many, 1)),
            lambda: tw.dense_fwd(m(many, 8), m(8, 8), None, m(many, 8), workspace=ws),
            lambda: tw.dense_fwd(m(few, 8), m(many, 8), None, m(few, many), workspace=ws),
            lambda: tw.dense_fwd(m(few, many), m(8, many), None, m(few, 8), workspace=ws),
            lambda: tw.dense_bwd(m(many, 8), m(8, 8), m(many, 8), m(8, 8), workspace=ws),
            lambda: tw.group_norm_fwd(m(many, 8), None, None, m(many, 8), None, None, positions=1, groups=1, workspace=ws),
            lambda: tw.group_norm_fwd(m(many, 8), None, None, m(many, 8), None, None, positions=many, groups=1, workspace=ws),
            lambda: tw.group_norm_fwd(m(few, 8), None, None, m(few, 8), None, None, positions=1, groups=many, workspace=ws),
            lambda: tw.group_norm_bwd(m(many, 8), m(many, 8), None, None, None, None, m(many, 8), None, None, positions=1,
                                      groups=1, workspace=ws)):
        with pytest.raises(ValueError, match="2\\^31"):
            bad()
    assert not calls
    tw.group_norm_fwd(m(2**33, 8), None, None, m(2**33, 8), None, None, positions=2**13, groups=1, workspace=ws)
    tw.act_dropout_fwd(m(2**31 - 1, 1), m(2**31 - 1, 1))
    assert [c[0] for c in calls] == ["el_group_norm_fwd", "el_act_dropout_fwd"]

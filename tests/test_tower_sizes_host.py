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

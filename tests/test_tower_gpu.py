"""The tower operators on the GPU against their plain 64-bit forms (tests/tower_plain.py, which
also derives the bounds), at the sizes, strides and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from tests import tower_plain as tp

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rows(rng, m, n, ld, dtype, scale=1.0, shift=0.0, at=0):
    """[m, n] values as columns at .. at+n-1 of rows ld wide, NaN around them."""
    full = torch.full((m, ld), float("nan"), dtype=DT[dtype])
    full[:, at:at + n] = torch.from_numpy(rng.normal(size=(m, n)) * scale + shift).to(DT[dtype])
    return full.to(DEV)[:, at:at + n]


def out(m, n, ld, dtype, at=0):
    return torch.full((m, ld), float("nan"), dtype=DT[dtype], device=DEV)[:, at:at + n]


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def gap_untouched(t):
    """The columns around a strided view still hold their NaN."""
    m, n = t.shape
    if m == 0:
        return True
    ld, at = t.stride(0), t.storage_offset()
    full = torch.as_strided(t, (m, ld), (ld, 1), 0).float()
    return bool(torch.isnan(full[:, :at]).all()) and bool(torch.isnan(full[:, at + n:]).all())


def make_drop(p, seed=0x1234_5678_9ABC_DEF0, offset=(3 << 32) + 5):
    return (elf.Dropout(p, seed, offset), seed, offset) if p is not None else (None, 0, 0)


# ------------------------------------------------------------------------- act_dropout
AD_CASES = [
    # M, N, ld, column offset, dtype, act, p, residual
    (1, 1, 1, 0, "f32", "gelu", 0.5, True),
    (1, 8, 8, 0, "bf16", "none", 0.25, False),
    (3, 7, 7, 0, "f16", "silu", 0.1, True),
    (64, 128, 128, 0, "bf16", "relu", 0.2, True),
    (33, 479, 512, 0, "f32", "silu", 0.3, False),
    (17, 257, 259, 1, "bf16", "gelu", 0.7, True),       # rows at odd addresses
    (5, 1001, 1003, 2, "f16", "gelu", None, True),
    (300, 65, 65, 0, "f32", "relu", 1.0, True),         # everything dropped
    (129, 1024, 1032, 0, "bf16", "gelu", 2.0**-16, False),
    (2500, 24, 24, 0, "f16", "silu", 0.999, False),
    (4, 9, 64, 3, "f32", "none", 0.0, False),
    (2050, 512, 512, 0, "bf16", "gelu", 0.1, True),     # several groups per thread
]


@pytest.mark.parametrize("case", AD_CASES, ids=lambda c: "-".join(map(str, c)))
def test_act_dropout(case):
    M, N, ld, at, dt, kind, p, res = case
    rng = np.random.default_rng(M * 1000 + N)
    x = rows(rng, M, N, ld, dt, 2.0, at=at)
    r = rows(rng, M, N, ld, dt, at=at) if res else None
    dy = rows(rng, M, N, ld, dt, at=at)
    y, dx = out(M, N, ld, dt, at), out(M, N, ld, dt, at)
    d, seed, offset = make_drop(p)
    elf.act_dropout_fwd(x, y, act=kind, dropout=d, residual=r)
    elf.act_dropout_bwd(dy, x if kind != "none" else None, dx, act=kind, dropout=d)
    f = tp.drop_factors(M, N, p, seed, offset) if p is not None else None
    tp.check(y, tp.act_dropout_fwd(np64(x), kind, f, np64(r), DT[dt]), "y")
    tp.check(dx, tp.act_dropout_bwd(np64(dy), np64(x), kind, f, DT[dt]), "dx")
    assert gap_untouched(y) and gap_untouched(dx)
    y2 = out(M, N, ld, dt, at)
    elf.act_dropout_fwd(x, y2, act=kind, dropout=d, residual=r)
    assert torch.equal(y, y2)


def test_act_dropout_mask_is_exactly_the_definition():
    M, N, p = 37, 203, 0.37
    x = torch.ones(M, N, device=DEV)
    y = torch.empty_like(x)
    for seed, offset in ((0, 0), (2**64 - 1, 2**64 - 1), (0x9E3779B97F4A7C15, 1 << 40)):
        elf.act_dropout_fwd(x, y, dropout=elf.Dropout(p, seed, offset))
        f = tp.drop_factors(M, N, p, seed, offset)
        assert ((np64(y) > 0) == (f > 0)).all()
        # the step on the device is added to the offset
        step = torch.tensor([5], dtype=torch.int64, device=DEV)
        elf.act_dropout_fwd(x, y, dropout=elf.Dropout(p, seed, offset, step))
        assert ((np64(y) > 0) == (tp.drop_factors(M, N, p, seed, offset + 5) > 0)).all()


def test_act_dropout_drops_infinities_and_nan():
    M, N, p = 16, 64, 0.5
    f = tp.drop_factors(M, N, p, 9, 9)
    x = torch.full((M, N), 2.0, device=DEV)
    bad = torch.from_numpy(f == 0).to(DEV)
    x[bad] = torch.tensor([float("inf"), float("-inf"), float("nan"), torch.finfo(torch.float32).min], device=DEV)[
        torch.arange(int(bad.sum()), device=DEV) % 4]
    y, dx = torch.empty_like(x), torch.empty_like(x)
    elf.act_dropout_fwd(x, y, dropout=elf.Dropout(p, 9, 9))
    elf.act_dropout_bwd(x, None, dx, dropout=elf.Dropout(p, 9, 9))
    want = torch.from_numpy(2.0 * f).float().to(DEV)
    assert torch.equal(y, want) and torch.equal(dx, want)


def test_act_dropout_empty_and_side_stream():
    e = torch.empty((0, 16), device=DEV)
    elf.act_dropout_fwd(e, torch.empty_like(e))
    x = torch.randn(513, 333, device=DEV)
    y, ref = torch.empty_like(x), torch.empty_like(x)
    elf.act_dropout_fwd(x, ref, act="gelu", dropout=elf.Dropout(0.3, 1))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    elf.act_dropout_fwd(x, y, act="gelu", dropout=elf.Dropout(0.3, 1), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, ref)


# ------------------------------------------------------------------------- dense
DENSE_CASES = [
    # M, K, N, extra stride, dtype, act, p, residual, pre
    (1, 1, 1, 0, "bf16", "gelu", 0.5, True, True),
    (1, 1024, 1024, 0, "bf16", "gelu", None, True, False),
    (1, 64, 40, 0, "f16", "silu", 0.25, False, True),
    (2, 479, 33, 33, "f16", "silu", 0.1, True, True),
    (16, 256, 512, 0, "bf16", "relu", None, False, False),
    (17, 520, 256, 8, "bf16", "silu", 0.5, True, True),
    (33, 31, 1001, 1, "bf16", "gelu", 0.3, True, True),   # odd rows of every operand
    (77, 512, 1024, 0, "f16", "silu", None, False, False),
    (129, 1024, 512, 0, "bf16", "gelu", 0.1, True, True),
    (256, 128, 256, 0, "bf16", "none", None, False, True),
    (300, 16, 1, 0, "bf16", "none", None, False, False),  # one logit per row
    (513, 200, 264, 24, "f16", "relu", 0.9, True, True),
    (1030, 256, 520, 0, "bf16", "gelu", 0.1, True, True),
    (64, 8, 2056, 0, "bf16", "relu", 1.0, True, True),
]


@pytest.mark.parametrize("case", DENSE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_dense_fwd(case):
    M, K, N, extra, dt, kind, p, res, keep = case
    rng = np.random.default_rng(M + 7 * K + 13 * N)
    x, w = rows(rng, M, K, K + extra, dt), rows(rng, N, K, K, dt, 1 / np.sqrt(K)).contiguous()
    bias = torch.from_numpy(rng.normal(size=N)).float().to(DEV) if M != 16 else None
    r = rows(rng, M, N, N + extra, dt) if res else None
    y, pre = out(M, N, N + extra, dt), out(M, N, N + extra, dt) if keep else None
    d, seed, offset = make_drop(p)
    elf.dense_fwd(x, w, bias, y, act=kind, dropout=d, residual=r, pre=pre)
    f = tp.drop_factors(M, N, p, seed, offset) if p is not None else None
    ry, ey, rz, ez = tp.dense_fwd(np64(x), np64(w), np64(bias), kind, f, np64(r), DT[dt])
    tp.check(y, (ry, ey), "y")
    assert gap_untouched(y)
    if keep:
        tp.check(pre, (rz, ez), "pre")
        assert gap_untouched(pre)
    y2 = out(M, N, N + extra, dt)
    elf.dense_fwd(x, w, bias, y2, act=kind, dropout=d, residual=r)
    assert torch.equal(y, y2), "not reproducible, or pre changes y"


@pytest.mark.parametrize("case", DENSE_CASES + [
    (4099, 72, 48, 0, "bf16", "gelu", 0.1, True, True),
    (2048, 256, 256, 0, "f16", "silu", None, True, True),
    (5000, 17, 9, 0, "bf16", "silu", 0.5, False, True),
], ids=lambda c: "-".join(map(str, c)))
def test_dense_bwd(case):
    M, K, N, extra, dt, kind, p, res, below = case
    rng = np.random.default_rng(3 * M + 5 * K + N)
    x, w = rows(rng, M, K, K + extra, dt), rows(rng, N, K, K, dt, 1 / np.sqrt(N)).contiguous()
    dz = rows(rng, M, N, N + extra, dt)
    dres = rows(rng, M, K, K + extra, dt) if res else None
    pre = rows(rng, M, K, K + extra, dt, 1.5) if below and kind != "none" else None
    dx, dzb = out(M, K, K + extra, dt), out(M, K, K + extra, dt) if below else None
    dw, db = torch.full((N, K), float("nan"), device=DEV), torch.full((N,), float("nan"), device=DEV)
    d, seed, offset = make_drop(p)
    elf.dense_bwd(x, w, dz, dw, db, dx=dx, dres=dres, dzb=dzb, pre=pre, act=kind, dropout=d)
    f = tp.drop_factors(M, K, p, seed, offset) if p is not None else None
    ref = tp.dense_bwd(np64(x), np64(w), np64(dz), np64(dres), np64(pre), kind, f, DT[dt])
    tp.check(dw, ref["dw"], "dw")
    tp.check(db, ref["db"], "db")
    tp.check(dx, ref["dx"], "dx")
    assert gap_untouched(dx)
    if below:
        tp.check(dzb, ref["dzb"], "dzb")
        assert gap_untouched(dzb)
    # the weight gradients alone, without db, from a workspace full of NaN: the same bits
    ws = torch.full((max(4, elf.dense_bwd_workspace_bytes(M, K, N) // 4),), float("nan"), device=DEV)
    dw2 = torch.empty_like(dw)
    elf.dense_bwd(x, w, dz, dw2, workspace=ws)
    assert torch.equal(dw, dw2)


def test_dense_empty_batch():
    x, w = torch.zeros((0, 24), dtype=torch.bfloat16, device=DEV), torch.ones((16, 24), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((0, 16), dtype=torch.bfloat16, device=DEV)
    elf.dense_fwd(x, w, None, y, act="gelu")
    dw, db = torch.full((16, 24), 7.0, device=DEV), torch.full((16,), 7.0, device=DEV)
    elf.dense_bwd(x, w, y, dw, db, dx=torch.empty_like(x))
    assert (dw == 0).all() and (db == 0).all()


def test_dense_nonfinite_rows_stay_in_their_rows():
    M, K, N = 70, 96, 72
    rng = np.random.default_rng(1)
    x, w = rows(rng, M, K, K, "bf16").contiguous(), rows(rng, N, K, K, "bf16").contiguous()
    y, y2 = torch.empty((M, N), dtype=torch.bfloat16, device=DEV), torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    elf.dense_fwd(x, w, None, y, act="silu")
    x2 = x.clone()
    x2[5], x2[69] = float("nan"), float("inf")
    elf.dense_fwd(x2, w, None, y2, act="silu")
    assert torch.isnan(y2[5].float()).all() and not torch.isfinite(y2[69].float()).all()
    ok = torch.ones(M, dtype=torch.bool, device=DEV)
    ok[5] = ok[69] = False
    assert torch.equal(y[ok], y2[ok])


# ------------------------------------------------------------------------- group norm
GN_CASES = [
    # B, S, C, G, ld, dtype, act, lengths, affine
    (1, 1, 1, 1, 1, "f32", "none", None, True),
    (5, 1, 512, 4, 512, "bf16", "gelu", None, True),        # layer-norm like rows
    (64, 26, 128, 8, 128, "bf16", "none", None, True),
    (37, 26, 128, 8, 136, "f16", "silu", "mixed", True),
    (9, 201, 96, 6, 96, "f32", "silu", "mixed", True),      # groups of 16 channels
    (7, 33, 30, 3, 31, "f32", "relu", "mixed", True),       # groups of 10 channels, odd rows
    (300, 3, 16, 16, 16, "bf16", "gelu", None, False),      # one channel per group
    (2, 2000, 64, 8, 64, "f16", "silu", "mixed", True),     # several chunks of positions
    (3, 700, 257, 1, 257, "f32", "gelu", "mixed", True),    # odd rows, one group
    (1, 5001, 24, 2, 24, "bf16", "none", None, True),
    (2, 40, 2304, 32, 2304, "bf16", "silu", "mixed", True),  # more than 256 vectors of channels
    (4, 17, 8, 1, 8, "f32", "none", "zero", True),
    (700, 2, 40, 5, 40, "f32", "silu", None, True),         # many samples per workgroup
]


@pytest.mark.parametrize("case", GN_CASES, ids=lambda c: "-".join(map(str, c)))
def test_group_norm(case):
    B, S, C, G, ld, dt, kind, masks, affine = case
    rng = np.random.default_rng(B + 3 * S + 7 * C)
    x = rows(rng, B * S, C, ld, dt, 1.5, 0.7)
    dy = rows(rng, B * S, C, ld, dt)
    ln = None
    if masks:
        v = rng.integers(0, S + 1, B) if masks == "mixed" else np.zeros(B, int)
        v[0], v[-1] = 0, (S if masks == "mixed" else 0)
        ln = torch.from_numpy(v.astype(np.int32)).to(DEV)
        pad = (torch.arange(S)[None, :] >= torch.from_numpy(v)[:, None]).reshape(-1).to(DEV)
        x[pad], dy[pad] = float("inf"), float("nan")        # padding is not read
    gm = torch.from_numpy(1 + 0.3 * rng.normal(size=C)).float().to(DEV) if affine else None
    bt = torch.from_numpy(0.3 * rng.normal(size=C)).float().to(DEV) if affine else None
    y, dx = out(B * S, C, ld, dt), out(B * S, C, ld, dt)
    nan = float("nan")
    mean, rstd = torch.full((B, G), nan, device=DEV), torch.full((B, G), nan, device=DEV)
    dg, db = torch.full((C,), nan, device=DEV), torch.full((C,), nan, device=DEV)
    kw = dict(positions=S, groups=G, act=kind, lengths=ln)
    elf.group_norm_fwd(x, gm, bt, y, mean, rstd, eps=1e-5, **kw)
    elf.group_norm_bwd(dy, x, gm, bt, mean, rstd, dx, dg, db, **kw)
    lens = None if ln is None else ln.cpu().numpy()
    X, D = (np.nan_to_num(np64(t), nan=0.0, posinf=0.0) for t in (x, dy))
    ry, ey, rm, rr = tp.gn_fwd(X, S, G, lens, np64(gm), np64(bt), 1e-5, kind, DT[dt])
    tp.check(mean, rm, "mean")
    tp.check(rstd, rr, "rstd")
    tp.check(y, (ry, ey), "y")
    ref = tp.gn_bwd(D, X, S, G, lens, np64(gm), np64(bt), np64(mean), np64(rstd), kind, DT[dt])
    tp.check(dx, ref["dx"], "dx")
    tp.check(dg, ref["dgamma"], "dgamma")
    tp.check(db, ref["dbeta"], "dbeta")
    assert gap_untouched(y) and gap_untouched(dx)
    # without the parameters' gradients, and again: the same bits
    dx2, dg2 = torch.empty_like(dx), torch.empty_like(dg)
    elf.group_norm_bwd(dy, x, gm, bt, mean, rstd, dx2, None, None, **kw)
    assert torch.equal(dx, dx2)
    elf.group_norm_bwd(dy, x, gm, bt, mean, rstd, dx2, dg2, None, **kw)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_group_norm_lengths_are_clamped_and_offsets_do_not_cancel():
    B, S, C, G = 3, 50, 32, 4
    x = (torch.randn(B * S, C, dtype=torch.float64) * 0.1 + 1000.0).float().to(DEV)  # a mean far from zero
    ln = torch.tensor([-7, 50, 2**31 - 1], dtype=torch.int32, device=DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty((B, G), device=DEV), torch.empty((B, G), device=DEV)
    elf.group_norm_fwd(x, None, None, y, mean, rstd, positions=S, groups=G, lengths=ln)
    ry, ey, rm, rr = tp.gn_fwd(np64(x), S, G, np.array([0, 50, 50]), None, None, 1e-5, "none", torch.float32)
    tp.check(mean, rm, "mean")
    assert (y[:S] == 0).all()
    # centred values: the spread is exact to a few steps although the mean is 1e4 spreads away
    assert np.max(np.abs(np64(rstd)[1:] / rr[0][1:] - 1)) < 1e-3
    assert float(rstd[0, 0]) == pytest.approx(1e-5 ** -0.5, rel=1e-6)


def test_gradients_match_differences_of_the_64_bit_forward():
    """<dx, d> against (L(x + h d) - L(x - h d)) / 2h with the forward in 64 bits."""
    rng = np.random.default_rng(8)
    M, K, N, h = 40, 48, 56, 1e-5
    x, w, co = rng.normal(size=(M, K)), rng.normal(size=(N, K)) / 7, rng.normal(size=(M, N))
    t = lambda a, dt=torch.bfloat16: torch.from_numpy(a).to(dt).to(DEV)  # noqa: E731
    xt, wt, ct = t(x), t(w), t(co)
    x, w, co = np64(xt), np64(wt), np64(ct)
    f = tp.drop_factors(M, N, 0.2, 11, 12)
    d = elf.Dropout(0.2, 11, 12)
    y, pre, dz, dx = (torch.empty((M, n), dtype=torch.bfloat16, device=DEV) for n in (N, N, N, K))
    dw = torch.empty((N, K), device=DEV)
    elf.dense_fwd(xt, wt, None, y, act="gelu", dropout=d, pre=pre)
    elf.act_dropout_bwd(ct, pre, dz, act="gelu", dropout=d)
    elf.dense_bwd(xt, wt, dz, dw, dx=dx)
    L = lambda a, b: float((tp.dense_fwd(a, b, None, "gelu", f, None, torch.float32)[0] * co).sum())  # noqa: E731
    for grad, dirn, diff in (
            (np64(dx), (dirx := rng.normal(size=x.shape)), (L(x + h * dirx, w) - L(x - h * dirx, w)) / (2 * h)),
            (np64(dw), (dirw := rng.normal(size=w.shape)), (L(x, w + h * dirw) - L(x, w - h * dirw)) / (2 * h))):
        # pre, dz and dx are each rounded once to bf16 (half a step 2^-8 of the value)
        assert abs((grad * dirn).sum() - diff) <= 3 * 2.0**-8 * np.abs(grad * dirn).sum()


# ------------------------------------------------------------------------- graph
def test_a_captured_layer_replays_with_another_mask_each_time():
    M, D, S, G = 130, 64, 5, 4
    rng = np.random.default_rng(2)
    x, w, dz = (rows(rng, m, D, D, "bf16").contiguous() for m in (M, D, M))
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    d = elf.Dropout(0.5, 77, 1000, step)
    E = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    f32 = torch.float32
    names = dict(y=E(M, D), pre=E(M, D), n=E(M, D), mean=E(M // S, G, dt=f32), rstd=E(M // S, G, dt=f32), dx=E(M, D),
                 dzb=E(M, D), dw=E(D, D, dt=f32), db=E(D, dt=f32), dn=E(M, D), dg=E(D, dt=f32), dbt=E(D, dt=f32))
    gm, bt = torch.ones(D, device=DEV), torch.zeros(D, device=DEV)
    ws = torch.empty(max(256, elf.dense_bwd_workspace_bytes(M, D, D), elf.group_norm_bwd_workspace_bytes(M // S, S, D, G),
                         elf.dense_fwd_workspace_bytes(M, D, D)), dtype=torch.uint8, device=DEV)

    def layer(o):
        elf.group_norm_fwd(x, gm, bt, o["n"], o["mean"], o["rstd"], positions=S, groups=G, act="silu", workspace=ws)
        elf.dense_fwd(o["n"], w, None, o["y"], act="gelu", dropout=d, residual=x, pre=o["pre"], workspace=ws)
        elf.dense_bwd(o["n"], w, dz, o["dw"], o["db"], dx=o["dx"], dzb=o["dzb"], pre=o["pre"], act="gelu", dropout=d,
                      dres=dz, workspace=ws)
        elf.group_norm_bwd(o["dx"], x, gm, bt, o["mean"], o["rstd"], o["dn"], o["dg"], o["dbt"], positions=S, groups=G,
                           act="silu", workspace=ws)

    layer(names)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer(names)
    seen = []
    for k in range(4):
        step.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        eager = {n: torch.full_like(t, float("nan")) for n, t in names.items()}
        layer(eager)
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(names[n], eager[n]), (k, n)
        seen.append(names["y"].clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


# ------------------------------------------------------------------------- every tile shape
@pytest.mark.parametrize("M,K,N", [
    (33_000, 40, 264),     # forward: 256 x 256 tiles with ragged edges
    (4_200, 72, 1_032),    # 128 x 128
    (2_200, 72, 520),      # 64 x 64
    (40_000, 24, 1),       # one column
])
def test_dense_fwd_tile_shapes(M, K, N):
    rng = np.random.default_rng(M)
    x, w = rows(rng, M, K, K, "bf16").contiguous(), rows(rng, N, K, K, "bf16", 1 / np.sqrt(K)).contiguous()
    bias = torch.from_numpy(rng.normal(size=N)).float().to(DEV)
    r, y, pre = rows(rng, M, N, N + 8, "bf16"), out(M, N, N + 8, "bf16"), out(M, N, N + 8, "bf16")
    d, seed, offset = make_drop(0.3)
    elf.dense_fwd(x, w, bias, y, act="gelu", dropout=d, residual=r, pre=pre)
    f = tp.drop_factors(M, N, 0.3, seed, offset)
    ry, ey, rz, ez = tp.dense_fwd(np64(x), np64(w), np64(bias), "gelu", f, np64(r), DT["bf16"])
    tp.check(y, (ry, ey), "y")
    tp.check(pre, (rz, ez), "pre")
    assert gap_untouched(y) and gap_untouched(pre)


@pytest.mark.parametrize("M,K,N", [
    (24_600, 1_000, 1_032),  # both products in 256 x 256 tiles
    (5_000, 1_032, 1_032),   # both in 128 x 128
    (4_200, 1_032, 136),     # data gradient 128 x 128, weight gradient 64 x 64
    (5_700, 520, 1_032),     # data gradient 64 x 64, weight gradient 128 x 128
    (33_000, 264, 72),       # data gradient 256 x 256, weight gradient 64 x 64
])
def test_dense_bwd_tile_shapes(M, K, N):
    rng = np.random.default_rng(M)
    x, w = rows(rng, M, K, K, "bf16").contiguous(), rows(rng, N, K, K, "bf16", 1 / np.sqrt(N)).contiguous()
    dz, dres, pre = rows(rng, M, N, N, "bf16").contiguous(), rows(rng, M, K, K, "bf16"), rows(rng, M, K, K, "bf16", 1.5)
    dx, dzb = out(M, K, K + 8, "bf16"), out(M, K, K + 8, "bf16")
    dw, db = torch.full((N, K), float("nan"), device=DEV), torch.full((N,), float("nan"), device=DEV)
    d, seed, offset = make_drop(0.3)
    elf.dense_bwd(x, w, dz, dw, db, dx=dx, dres=dres, dzb=dzb, pre=pre, act="silu", dropout=d)
    ref = tp.dense_bwd(np64(x), np64(w), np64(dz), np64(dres), np64(pre), "silu", tp.drop_factors(M, K, 0.3, seed, offset),
                       DT["bf16"])
    for name, got in (("dw", dw), ("db", db), ("dx", dx), ("dzb", dzb)):
        tp.check(got, ref[name], name)
    assert gap_untouched(dx) and gap_untouched(dzb)


@pytest.mark.parametrize("B,S,C,G,dt,kind", [
    (33, 1, 8, 1, "f32", "silu"), (33, 1, 8, 4, "bf16", "none"), (20, 2, 512, 64, "f16", "gelu"), (21, 10, 64, 16, "f32", "silu"),
    (20, 30, 32, 16, "bf16", "silu"), (10, 30, 128, 16, "f32", "gelu"), (9, 8, 512, 512, "f32", "none"),
    (50, 20, 96, 6, "bf16", "gelu"), (40, 64, 24, 1, "f32", "silu"), (33, 60, 48, 3, "f16", "relu"), (12, 33, 320, 32, "bf16", "silu"),
    (5, 3, 1000, 8, "f32", "gelu"), (2, 1, 4096, 4096, "f32", "none"), (3, 1, 5000, 1000, "bf16", "silu"),
])
def test_group_norm_forms(B, S, C, G, dt, kind):
    """One wavefront per sample or several samples in one, one workgroup, chunks; groups inside
    vectors, of whole vectors, across them."""
    rng = np.random.default_rng(C + S)
    x, dy = rows(rng, B * S, C, C, dt, 1.5, 0.7).contiguous(), rows(rng, B * S, C, C, dt).contiguous()
    gm, bt = (torch.from_numpy(a + 0.3 * rng.normal(size=C)).float().to(DEV) for a in (1, 0))
    y, dx = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    mean, rstd = torch.empty((B, G), device=DEV), torch.empty((B, G), device=DEV)
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    eps = 0.1  # groups of one or two values: keeps rstd and its cancellations moderate
    elf.group_norm_fwd(x, gm, bt, y, mean, rstd, positions=S, groups=G, eps=eps, act=kind)
    elf.group_norm_bwd(dy, x, gm, bt, mean, rstd, dx, dg, db, positions=S, groups=G, act=kind)
    ry, ey, rm, rr = tp.gn_fwd(np64(x), S, G, None, np64(gm), np64(bt), eps, kind, DT[dt])
    tp.check(mean, rm, "mean")
    tp.check(rstd, rr, "rstd")
    tp.check(y, (ry, ey), "y")
    ref = tp.gn_bwd(np64(dy), np64(x), S, G, None, np64(gm), np64(bt), np64(mean), np64(rstd), kind, DT[dt])
    tp.check(dx, ref["dx"], "dx")
    tp.check(dg, ref["dgamma"], "dgamma")
    tp.check(db, ref["dbeta"], "dbeta")


def test_rows_past_32_bit_offsets():
    """Row strides of 2^20 elements: the last rows of 2300 lie past 2^32 bytes."""
    M, K, N, ld = 2_300, 64, 72, 1 << 20
    big = torch.empty((M, ld), dtype=torch.bfloat16, device=DEV)
    at = {"x": 0, "dz": 100, "y": 200, "pre": 300, "dx": 400, "dres": 500, "dzb": 600, "gn": 700}
    view = lambda n, c: big[:, at[n]:at[n] + c]  # noqa: E731
    g = torch.Generator(DEV).manual_seed(5)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    src = {n: rnd(M, c) for n, c in (("x", K), ("dz", N), ("dres", K))}
    for n, t in src.items():
        view(n, t.shape[1]).copy_(t)
    w, d = rnd(N, K), elf.Dropout(0.2, 3)
    y, pre, dx, dzb = (torch.empty(M, c, dtype=torch.bfloat16, device=DEV) for c in (N, N, K, K))
    dw, dw2 = torch.empty(N, K, device=DEV), torch.empty(N, K, device=DEV)
    elf.dense_fwd(src["x"], w, None, y, act="gelu", dropout=d, pre=pre)
    elf.dense_fwd(view("x", K), w, None, view("y", N), act="gelu", dropout=d, pre=view("pre", N))
    assert torch.equal(y, view("y", N)) and torch.equal(pre, view("pre", N))
    elf.dense_bwd(src["x"], w, src["dz"], dw, dx=dx, dres=src["dres"], dzb=dzb, pre=src["x"], act="silu", dropout=d)
    elf.dense_bwd(view("x", K), w, view("dz", N), dw2, dx=view("dx", K), dres=view("dres", K), dzb=view("dzb", K),
                  pre=view("x", K), act="silu", dropout=d)
    assert torch.equal(dw, dw2) and torch.equal(dx, view("dx", K)) and torch.equal(dzb, view("dzb", K))
    elf.act_dropout_fwd(src["x"], dx, act="gelu", dropout=d)
    elf.act_dropout_fwd(view("x", K), view("dx", K), act="gelu", dropout=d)
    assert torch.equal(dx, view("dx", K))
    for S in (23, 1150):
        st = [torch.empty(M // S, 4, device=DEV) for _ in range(4)]
        elf.group_norm_fwd(src["x"], None, None, dx, st[0], st[1], positions=S, groups=4)
        elf.group_norm_fwd(view("x", K), None, None, view("gn", K), st[2], st[3], positions=S, groups=4)
        assert torch.equal(dx, view("gn", K)) and torch.equal(st[0], st[2]) and torch.equal(st[1], st[3])


def test_calls_follow_the_given_stream_and_the_current_one():
    M, K, N = 700, 128, 136
    x, w, dz = (torch.randn(*s, device=DEV).bfloat16() for s in ((M, K), (N, K), (M, N)))
    want = None
    side = torch.cuda.Stream()
    for how in ("default", "given", "current"):
        y, dw, dx = torch.empty(M, N, device=DEV).bfloat16(), torch.empty(N, K, device=DEV), torch.empty_like(x)
        ws = torch.empty(elf.dense_bwd_workspace_bytes(M, K, N), dtype=torch.uint8, device=DEV)
        kw = dict(stream=side) if how == "given" else {}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side) if how == "current" else torch.cuda.stream(None):
            elf.dense_fwd(x, w, None, y, act="silu", **kw)
            elf.dense_bwd(x, w, dz, dw, dx=dx, workspace=ws, **kw)
        torch.cuda.current_stream().wait_stream(side)
        got = (y.clone(), dw.clone(), dx.clone())
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(want, got)), how

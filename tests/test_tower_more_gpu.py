"""More sizes of the tower operators on the GPU, against the plain 64-bit forms and bounds of
tests/tower_plain.py: the kernel forms and loops that tests/test_tower_gpu.py's sizes do not reach."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from tests import test_tower_gpu as base
from tests import tower_plain as tp

pytestmark = pytest.mark.gpu
DEV = "cuda"

# more samples than 512 workgroups' worth: one workgroup has a sample's statistics
WHOLE = [
    # B, S, C, G, ld, dtype, act, lengths, affine
    (300, 40, 520, 8, 520, "bf16", "silu", "mixed", True),   # groups across vectors
    (260, 9, 1888, 32, 1888, "bf16", "gelu", None, True),    # wide: one row of threads
    (260, 70, 257, 1, 259, "f32", "silu", "mixed", True),    # odd rows, one group
    (257, 45, 400, 40, 400, "f16", "gelu", "mixed", False),  # groups of 10 channels
    (258, 200, 128, 128, 128, "f32", "none", "mixed", True),  # one channel per group
    (520, 30, 2048, 1, 2048, "f16", "none", "zero", True),
]


@pytest.mark.parametrize("case", WHOLE, ids=lambda c: "-".join(map(str, c)))
def test_group_norm_whole_samples(case):
    base.test_group_norm(case)


def test_dense_bwd_of_the_longest_batch():
    """2^31 - 1 rows: the last slice of the reduction ends where a 32-bit sum would have passed 2^31,
    and no row behind the last is read.  A few rows count, the others are zeros."""
    M, K, N = 2**31 - 1, 8, 8
    x = torch.zeros((M + 1, K), dtype=torch.bfloat16, device=DEV)
    dz = torch.zeros((M + 1, N), dtype=torch.bfloat16, device=DEV)
    at = [0, 1, 63, 2**23 - 1, 2**23, 2**30, 2**31 - 2**23 - 1, 2**31 - 2**23, M - 64, M - 1]
    rng = np.random.default_rng(0)
    xs, zs = rng.integers(-8, 9, (len(at), K)), rng.integers(-8, 9, (len(at), N))
    x[at], dz[at] = (torch.from_numpy(v).to(torch.bfloat16).to(DEV) for v in (xs, zs))
    x[M], dz[M] = float("nan"), float("nan")  # behind the last row
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    elf.dense_bwd(x[:M], w=torch.ones(N, K, dtype=torch.bfloat16, device=DEV), dz=dz[:M], dw=dw, db=db, workspace=ws)
    assert (dw.cpu().numpy() == zs.T @ xs).all() and (db.cpu().numpy() == zs.sum(0)).all()


@pytest.mark.parametrize("B,S,C,G,dt", [
    (70, 26, 128, 8, "bf16"), (70, 26, 128, 8, "f32"), (40, 30, 128, 32, "f32"), (33, 1, 64, 1, "f16"), (50, 5, 32, 4, "f32"),
    (20, 40, 96, 6, "f32"), (21, 33, 30, 3, "bf16"), (9, 20, 520, 5, "f32"), (3, 2000, 64, 8, "f32"), (2, 900, 257, 1, "f16"),
    (6, 1, 40, 40, "f32"), (4, 1, 64, 64, "f32"),
])
def test_group_norm_gradients_do_not_see_an_offset(B, S, C, G, dt):
    """x and mean moved by one number, every value exact before and after: the centred values are the
    same bits, and so are the gradients (all forms; also where a group is one value and xh is 0)."""
    g = torch.Generator(DEV).manual_seed(B + C)
    move = {"f32": 4096.0, "f16": 1024.0, "bf16": 240.0}[dt]
    x = torch.randint(0, 16, (B * S, C), generator=g, device=DEV).to(base.DT[dt])
    dy = torch.randn(B * S, C, generator=g, device=DEV).to(base.DT[dt])
    gm, bt = (torch.randn(C, generator=g, device=DEV) for _ in range(2))
    mean = torch.randint(0, 128, (B, G), generator=g, device=DEV) / 8.0
    if C == G and S == 1:
        mean = x.float()
    rstd = torch.rand(B, G, generator=g, device=DEV) + 0.5
    got = []
    for m in (0.0, move):
        dx, dg, db = torch.full_like(x, float("nan")), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        elf.group_norm_bwd(dy, x + m, gm, bt, mean + m, rstd, dx, dg, db, positions=S, groups=G, act="silu")
        got.append((dx, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    if C == G and S == 1:  # xh = 0, dh = avg dh: nothing but the rounding of du gamma (|du| <= 1.1 |dy|)
        assert (got[1][1] == 0).all()
        assert (got[1][0].abs() <= 4 * 2.0**-24 * (dy * gm).abs() * rstd).all()


def test_group_norm_rows_of_the_largest_batch():
    """Every pooled vector of 262144 samples of 26 tables as a row (S = 1, one group): the same bits as
    in two halves, rows against the plain form, parameter gradients against sums in 64 bits."""
    B, C, kw = 26 * 262144, 128, dict(positions=1, groups=1)
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.empty(B, C, dtype=torch.bfloat16, device=DEV).normal_(0.5, 1.5, generator=g)
    dy = torch.empty(B, C, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    gm, bt = (torch.randn(C, generator=g, device=DEV) for _ in range(2))
    y, dx, y2, dx2 = (torch.full_like(x, float("nan")) for _ in range(4))
    st, st2 = (torch.full((2, B, 1), float("nan"), device=DEV) for _ in range(2))
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    elf.group_norm_fwd(x, gm, bt, y, st[0], st[1], act="silu", **kw)
    elf.group_norm_bwd(dy, x, gm, bt, st[0], st[1], dx, dg, db, act="none", **kw)
    for h in (slice(0, B // 2), slice(B // 2, B)):
        elf.group_norm_fwd(x[h], gm, bt, y2[h], st2[0, h], st2[1, h], act="silu", **kw)
        elf.group_norm_bwd(dy[h], x[h], gm, bt, st2[0, h], st2[1, h], dx2[h], None, None, act="none", **kw)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(st, st2)
    for at in (0, B // 2 - 50, B - 100):
        h, n = slice(at, at + 100), base.np64
        ry, ey, rm, rr = tp.gn_fwd(n(x[h]), 1, 1, None, n(gm), n(bt), 1e-5, "silu", torch.bfloat16)
        tp.check(y[h], (ry, ey), "y")
        ref = tp.gn_bwd(n(dy[h]), n(x[h]), 1, 1, None, n(gm), n(bt), n(st[0, h]), n(st[1, h]), "none", torch.bfloat16)
        tp.check(dx[h], ref["dx"], "dx")
    want, size = (torch.zeros(2, C, dtype=torch.float64, device=DEV) for _ in range(2))
    for at in range(0, B, 1 << 19):
        h = slice(at, at + (1 << 19))
        d = dy[h].double()
        q = d * (x[h].double() - st[0, h].double()) * st[1, h].double()
        want += torch.stack([q.sum(0), d.sum(0)])
        size += torch.stack([q.abs().sum(0), d.abs().sum(0)])
    # 416 samples behind each other in a thread, then joins of at most 64 additions; xh within 4 steps
    assert ((torch.stack([dg, db]).double() - want).abs() <= 512 * 2.0**-24 * size).all()


# ------------------------------------------------------------------------- dense layer, every tile shape
FWD = [
    # M, K, N, extra row stride: L, M and S tiles; whole vectors, then operands that are copied first
    (33_000, 40, 264, 8), (4_200, 72, 1_032, 8), (2_200, 72, 520, 0), (40_000, 24, 1, 8),
    (33_000, 43, 257, 5), (4_099, 479, 1_001, 33), (2_200, 71, 523, 1), (2_200, 72, 520, 3),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N,extra", FWD)
def test_dense_fwd_tiles(M, K, N, extra, dt):
    rng = np.random.default_rng(M + K)
    x, w = base.rows(rng, M, K, K + extra, dt), base.rows(rng, N, K, K, dt, 1 / np.sqrt(K)).contiguous()
    bias = torch.from_numpy(rng.normal(size=N)).float().to(DEV)
    r, y, pre = (base.rows(rng, M, N, N + extra, dt), base.out(M, N, N + extra, dt), base.out(M, N, N + extra, dt))
    d, seed, offset = base.make_drop(0.3)
    n = base.np64
    ws = torch.full((elf.dense_fwd_workspace_bytes(M, K, N) // 4,), float("nan"), device=DEV)
    elf.dense_fwd(x, w, bias, y, act="silu", dropout=d, residual=r, pre=pre, workspace=ws)
    ry, ey, rz, ez = tp.dense_fwd(n(x), n(w), n(bias), "silu", tp.drop_factors(M, N, 0.3, seed, offset), n(r), base.DT[dt])
    tp.check(y, (ry, ey), "y")
    tp.check(pre, (rz, ez), "pre")
    assert base.gap_untouched(y) and base.gap_untouched(pre)


BWD = [
    # M, K, N, extra: both products L, both M, M and S, S and M, L and S; then copied operands
    (24_600, 1_000, 1_032, 0), (5_000, 1_032, 1_032, 0), (4_200, 1_032, 136, 8), (5_700, 520, 1_032, 0),
    (33_000, 264, 72, 8), (33_000, 261, 70, 3), (5_001, 1_031, 1_030, 1), (4_099, 517, 260, 0), (4_099, 512, 257, 7),
]


@pytest.mark.parametrize("M,K,N,extra,dt", [(*c, "f16") for c in BWD] + [(*c, "bf16") for c in BWD[5:]])
def test_dense_bwd_tiles(M, K, N, extra, dt):
    rng = np.random.default_rng(M + K)
    x, w = base.rows(rng, M, K, K + extra, dt), base.rows(rng, N, K, K, dt, 1 / np.sqrt(N)).contiguous()
    dz, dres, pre = (base.rows(rng, M, c, c + extra, dt, s) for c, s in ((N, 1.0), (K, 1.0), (K, 1.5)))
    dx, dzb = base.out(M, K, K + extra, dt), base.out(M, K, K + extra, dt)
    dw, db = torch.full((N, K), float("nan"), device=DEV), torch.full((N,), float("nan"), device=DEV)
    d, seed, offset = base.make_drop(0.3)
    n = base.np64
    ws = torch.full((elf.dense_bwd_workspace_bytes(M, K, N) // 4,), float("nan"), device=DEV)
    elf.dense_bwd(x, w, dz, dw, db, dx=dx, dres=dres, dzb=dzb, pre=pre, act="gelu", dropout=d, workspace=ws)
    ref = tp.dense_bwd(n(x), n(w), n(dz), n(dres), n(pre), "gelu", tp.drop_factors(M, K, 0.3, seed, offset), base.DT[dt])
    for name, got in (("dw", dw), ("db", db), ("dx", dx), ("dzb", dzb)):
        tp.check(got, ref[name], name)
    assert base.gap_untouched(dx) and base.gap_untouched(dzb)
    dw2 = torch.empty_like(dw)
    if M < 20_000:  # (shape L has other slices without dx)
        elf.dense_bwd(x, w, dz, dw2, workspace=ws)
        assert torch.equal(dw, dw2)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(33_000, 40, 264), (4_200, 72, 1_032), (2_200, 72, 520), (4_099, 479, 1_001)])
def test_non_finite_rows_stay_in_their_rows_in_every_tile_shape(M, K, N, dt):
    rng = np.random.default_rng(N)
    x, w = base.rows(rng, M, K, K, dt).contiguous(), base.rows(rng, N, K, K, dt).contiguous()
    bad = [0, 5, 63, 64, 127, 255, 256, M // 2, M - 2, M - 1]
    x2 = x.clone()
    x2[bad] = torch.tensor([float("nan"), float("inf")], device=DEV).to(base.DT[dt]).repeat(5)[:, None]
    ok = torch.ones(M, dtype=torch.bool, device=DEV)
    ok[bad] = False
    y, y2 = torch.empty(M, N, dtype=base.DT[dt], device=DEV), torch.empty(M, N, dtype=base.DT[dt], device=DEV)
    elf.dense_fwd(x, w, None, y, act="silu")
    elf.dense_fwd(x2, w, None, y2, act="silu")
    assert torch.equal(y[ok], y2[ok]) and torch.isfinite(y[ok].float()).all()
    assert not torch.isfinite(y2[bad].float()).any()
    # the data gradient's rows likewise
    dw, dx, dx2 = torch.empty(K, N, device=DEV), torch.empty_like(y), torch.empty_like(y)
    wt = w.t().contiguous()
    elf.dense_bwd(y, wt, x, dw, dx=dx)
    elf.dense_bwd(y, wt, x2, dw, dx=dx2)
    assert torch.equal(dx[ok], dx2[ok]) and torch.isnan(dx2[bad[0]].float()).all()


# ------------------------------------------------------------------------- group norm, several samples a workgroup in turn
LOOPS = [
    # B, S, C, G, ld, dtype, act, lengths, affine: more samples than one round of workgroups takes
    (2501, 26, 128, 8, 128, "bf16", "silu", "mixed", True),    # wavefronts, eight vectors a lane
    (2501, 26, 128, 32, 128, "f16", "gelu", "mixed", True),    # per-channel sums, 16 bits
    (2501, 26, 128, 32, 136, "f32", "silu", None, True),
    (2501, 26, 128, 8, 128, "f32", "none", "mixed", False),
    (262_403, 1, 8, 1, 8, "bf16", "silu", "mixed", True),      # one lane a sample
    (17_001, 3, 64, 64, 64, "f16", "none", None, True),
    (4501, 10, 30, 3, 31, "bf16", "silu", "mixed", True),      # one wavefront of threads, partial vectors
    (4501, 20, 96, 6, 96, "f16", "gelu", None, True),
    (1101, 40, 96, 4, 96, "f32", "silu", "mixed", True),       # 256 threads
    (3500, 1, 600, 50, 600, "bf16", "silu", None, True),       # three samples a workgroup
    (500, 1, 2304, 9, 2304, "f32", "gelu", "mixed", True),     # 288 threads
    (500, 2, 2040, 1, 2048, "f16", "silu", "mixed", True),     # 510 threads
]


@pytest.mark.parametrize("case", LOOPS, ids=lambda c: "-".join(map(str, c)))
def test_group_norm_loops(case):
    base.test_group_norm(case)


@pytest.mark.parametrize("B,S,C,G,dt,outlier", [
    (513, 4000, 1040, 1040, "bf16", 1000.0),  # one chunk a sample: a thread sums 4000 positions
    (513, 4000, 1040, 65, "bf16", 1000.0),
    (2, 90_000, 64, 64, "f32", 3000.0),       # chunks of positions
    (513, 4000, 1040, 1040, "bf16", 0.5),     # and none
])
def test_group_norm_statistics_behind_a_large_first_position(B, S, C, G, dt, outlier):
    """Histories whose first position is far from all others: mean and rstd of a few samples against 64 bits."""
    g = torch.Generator(DEV).manual_seed(S)
    x = torch.empty(B * S, C, dtype=base.DT[dt], device=DEV).normal_(0.5, 1.0, generator=g)
    x[::S] = x[::S] + outlier
    y, mean, rstd = torch.empty_like(x), torch.empty(B, G, device=DEV), torch.empty(B, G, device=DEV)
    elf.group_norm_fwd(x, None, None, y, mean, rstd, positions=S, groups=G)
    for b in (0, B // 2, B - 1):
        v = x[b * S:(b + 1) * S].double().view(S, G, C // G)
        m = v.mean((0, 2))
        var = ((v - m[:, None]) ** 2).mean((0, 2))
        want = (var + 1e-5).rsqrt()
        # sums in fp32 of n positions a thread, n / 2 half steps for each of the sums of values and of
        # squares (four positions are added at a time), and trees behind them
        n = S if B > 2 else S // 16
        bound = (n / 2 + 64) * 2.0**-24
        assert ((mean[b].double() - m).abs() <= bound * v.abs().mean((0, 2))).all()
        assert ((rstd[b].double() / want - 1).abs() <= bound).all(), float((rstd[b].double() / want - 1).abs().max())

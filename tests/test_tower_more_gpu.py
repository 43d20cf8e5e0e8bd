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

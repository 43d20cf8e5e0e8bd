"""More of the residual block's operators on the GPU: the largest batches, and sums that have to be exact."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from tests import block_plain as bp
from tests import tower_plain as tp
from tests.test_block_gpu import norm_case
from tests.test_tower_gpu import DEV, DT, gap_untouched, np64, out

pytestmark = pytest.mark.gpu


def test_block_norm_shared_gates_of_more_than_2_to_the_30_rows():
    """M + gate_rows passes 2^31; two gate rows, the second of one row.  Small whole numbers: exact."""
    M, C = (1 << 30) + 3, 1
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dy, f, df, gate, dgate = z(M, C), z(M, C), z(M, C), z(2, C), z(2, C)
    f.fill_(1.0)
    dy[::65537] = 1.0
    dy[-1] = 4.0
    gate[0], gate[1] = 2.0, 3.0
    ones = -(-M // 65537)  # rows of dy that hold 1 (the last is not one of them)
    assert (M - 1) % 65537 != 0
    nm = elf.BlockNorm(C, post="none", pre="rms", gate_rows=M - 1)
    dgamma, dbeta = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    elf.block_norm_bwd(nm, None, None, dy=dy, f=f, gate=gate, df=df, dgate=dgate, dpost_gamma=dgamma, dpost_beta=dbeta)
    assert dgamma.item() == dbeta.item() == 2 * ones + 12
    assert torch.equal(dgate.cpu(), torch.tensor([[float(ones)], [4.0]]).bfloat16())
    assert bool((df[:-1] == 2 * dy[:-1]).all()) and df[-1].item() == 12.0


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,gr,C", [(37, 1, 64), (37, 1, 33), (40_000, 1, 24), (44, 4, 64), (44, 4, 33), (6_000, 3_000, 40),
                                    (70_000, 70_000, 16), (3_000, 3, 1024)])
def test_block_norm_open_and_closed_sigmoid_gates(M, gr, C, dt):
    """dgate = s (1 - s) sum over its rows of D t and df = s D, relative to themselves, at gates from far
    closed to far open: each in a row of its own, inside a slot's run, across two slots and across many.
    D t is 1 in every row, so its sums are exact.

    Bounds, u = 2^-24: the tail t = sigmoid(-|v|) is off by (4 + 2 |v|) u of itself (block_plain), t (1 - t)
    by one step more and by its product with the sum, 1 - t by (5 + 2 |v|) u; below 2^-126 it may be 0."""
    U, R = 2.0**-24, -(-M // gr)
    v = [0.0, 1.0, 3.0, 6.0, 9.0, 12.0, 15.0, 17.0, 18.0, 25.0, 40.0, 80.0, 200.0, float("inf")]
    v = torch.tensor(v + [-a for a in v])
    gate = v[torch.arange(R * C) % v.numel()].view(R, C).to(DT[dt]).to(DEV)
    ones = torch.ones((M, C), dtype=DT[dt], device=DEV)
    df, dgate = torch.empty_like(ones), torch.empty_like(gate)
    nm = elf.BlockNorm(C, post="none", gate_act="sigmoid", gate_rows=gr)
    elf.block_norm_bwd(nm, None, None, dy=ones, f=ones, gate=gate, df=df, dgate=dgate)
    w = gate.double().cpu()
    count = torch.full((R, 1), float(gr), dtype=torch.float64)
    count[-1] = M - (R - 1) * gr
    f = torch.finfo(DT[dt])
    store = lambda a: a * (f.eps / 2) * (1 + 2 * f.eps) + f.smallest_normal * f.eps / 2  # noqa: E731
    at = 2 * w.abs().clamp(max=100.0)
    want = torch.sigmoid(w) * torch.sigmoid(-w) * count
    err = (dgate.cpu().double() - want).abs()
    assert bool((err <= (7 + at) * U * want + count * 2.0**-126 + store(want)).all()), (err / want).max()
    want = torch.sigmoid(w).repeat_interleave(gr, 0)[:M]
    err = (df.cpu().double() - want).abs()
    assert bool((err <= (5 + at.repeat_interleave(gr, 0)[:M]) * U * want + 2.0**-126 + store(want)).all())


def test_block_norm_follows_a_parameter_whose_storage_was_replaced():
    M, C = 5, 256
    x = torch.randn((M, C), device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    gamma = torch.ones(C, device=DEV)
    nm, h, want = elf.BlockNorm(C, pre_gamma=gamma), torch.empty_like(x), torch.empty_like(x)
    elf.block_norm_fwd(nm, x, None, h)
    gamma.data = torch.linspace(-2, 2, C, device=DEV)
    junk = torch.full((C,), 77.0, device=DEV)  # (takes the old storage)
    elf.block_norm_fwd(nm, x, None, h)
    elf.block_norm_fwd(elf.BlockNorm(C, pre_gamma=gamma.clone()), x, None, want)
    assert torch.equal(h, want) and bool((junk == 77.0).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_ckpt_activations_of_magnitudes_that_round_to_infinity(dt):
    """fp32's largest magnitudes stand for infinities once packed (2^128): the activations' values there
    are those of act_dropout_fwd on the kept values, GELU's 0 below."""
    top = torch.finfo(torch.float32).max
    x = torch.tensor([top, -top, 3.3e38, -3.3e38, -1e30, -100.0, 0.0, 1.0] * 4, device=DEV).view(1, 32)
    ck = elf.ckpt_pack(x, elf.Checkpoint(1, 32, DEV))
    kept = elf.ckpt_act_dropout_fwd(ck, torch.empty_like(x))
    # (3.3e38 too: 3.3e38 / 2^120 = 248.3 lies above the middle of e4m3's 240 and 256, and 256 * 2^120 = 2^128)
    assert bool(kept[0, 0:4:2].isposinf().all()) and bool(kept[0, 1:4:2].isneginf().all()) and bool(kept[0, 4:8].isfinite().all())
    for act in ("relu", "gelu"):
        y = elf.ckpt_act_dropout_fwd(ck, torch.empty((1, 32), dtype=DT[dt], device=DEV), act=act)
        want = elf.act_dropout_fwd(kept, torch.empty_like(x), act=act).to(DT[dt])
        assert torch.equal(y, want), (act, y[0, :8], want[0, :8])
        assert bool(y[0, 0].isposinf()) and y[0, 1].item() == 0.0


def test_fp16_magnitudes_that_round_to_2_to_the_16_in_8_bits():
    """63488 lies in the middle of e4m3's 240 and 256 times 2^8 and goes to the even one: 2^16, kept as it
    is, infinity in fp16 and nowhere else."""
    M, K, N = 40, 64, 32
    x = torch.ones((M, K), dtype=torch.float16, device=DEV)
    x[3, 5], x[3, 6], x[7, 40], x[9, 33] = 63488.0, 63456.0, -65504.0, 61440.0
    ck = elf.ckpt_pack(x, elf.Checkpoint(M, K, DEV))
    y = elf.ckpt_act_dropout_fwd(ck, torch.empty((M, K), device=DEV))
    assert y[3, 5:7].tolist() == [65536.0, 61440.0] and y[7, 40].item() == -65536.0 and y[9, 33].item() == 61440.0
    for dt in (torch.float16, torch.bfloat16):
        y = elf.ckpt_act_dropout_fwd(ck, torch.empty((M, K), dtype=dt, device=DEV))
        w, dz = torch.zeros((N, K), dtype=dt, device=DEV), torch.full((M, N), 2.0**-6, dtype=dt, device=DEV)
        dw = torch.empty((N, K), device=DEV)
        elf.dense_bwd_ckpt(ck, w, dz, dw)
        inf = dt is torch.float16
        assert y.isinf().nonzero().tolist() == ([[3, 5], [7, 40]] if inf else [])
        cols = sorted(set(torch.isinf(dw).nonzero()[:, 1].tolist()))
        assert cols == ([5, 40] if inf else []) and not bool(dw.isnan().any())
        if not inf:
            # row 3's block has the scale 2^8, so its ones are kept as 1, as all are: 2^-6 (39 + 2^16)
            assert bool((dw[:, 5] == (39 + 65536.0) / 64).all()) and bool((dw[:, 40] == (39 - 65536.0) / 64).all())


# ------------------------------------------------------------------------- sums over rows, exactly
def whole(g, m, n, ld, dt, lo=-2, hi=2):
    """Whole numbers in columns of rows ld wide, NaN behind them."""
    full = torch.full((m, ld), float("nan"), dtype=DT[dt], device=DEV)
    full[:, :n] = torch.randint(lo, hi + 1, (m, n), device=DEV, generator=g).to(DT[dt])
    return full[:, :n]


EXACT = [
    # M, C, extra columns, dtype, gate_rows (None: no gate), betas
    # a gate row to each row, several rows to a slot, the last step cut
    (40_001, 128, 0, "bf16", 1, False), (40_001, 128, 0, "bf16", 1, True), (10_007, 479, 2, "f16", 1, True),
    (10_007, 479, 1, "f16", 1, False), (7_001, 512, 0, "f32", 1, True), (7_001, 512, 0, "f32", 1, False),
    (200_003, 16, 0, "bf16", 1, True), (200_003, 16, 0, "f32", None, False), (200_003, 13, 0, "bf16", None, True),
    (60_001, 64, 0, "f16", None, False), (30_011, 200, 0, "bf16", 1, True), (20_011, 256, 8, "f32", None, True),
    (9_001, 1024, 0, "bf16", 1, False), (9_001, 1024, 0, "bf16", 1, True), (9_001, 1000, 0, "f32", 1, False),
    (5_003, 2048, 0, "bf16", 1, True), (3_001, 4096, 0, "f16", 1, False), (2_003, 8192, 0, "bf16", None, True),
    (1_201, 16_384, 0, "bf16", 1, True), (700, 32_768, 0, "f16", None, False),
    # gate rows shared: within a slot's run, across slots, across very many
    (70_001, 16, 0, "f32", 26, True), (70_000, 24, 1, "bf16", 26, True), (30_000, 128, 0, "f16", 29_999, True),
    (40_000, 64, 0, "f32", 40_000, True), (100_003, 8, 0, "bf16", 2, True), (426_062, 128, 0, "bf16", 26, False),
    (65_536, 16, 0, "bf16", 65_536, False), (300_000, 40, 0, "f32", 7, True), (9_001, 1000, 0, "bf16", 50, True),
    (9_001, 1024, 0, "bf16", 3, False), (9_001, 1024, 0, "f16", 9_001, False), (5_003, 4096, 0, "bf16", 11, True),
    (2_003, 8200, 0, "f16", 5, True), (30_001, 1001, 0, "bf16", 21, True), (100_003, 32, 0, "f32", 500, False),
]


@pytest.mark.parametrize("case", EXACT, ids=lambda c: "-".join(map(str, c)))
def test_block_norm_sums_over_rows_are_exact(case):
    """Whole numbers so small that no sum passes 2^24: every order of additions gives the same bits, and a
    row that is dropped or taken twice shows.  (At most 24 a term, for 426062 rows 1.03e7.)"""
    M, C, ex, dt, gr, beta = case
    g = torch.Generator(DEV).manual_seed(M + C)
    R, ld = -(-M // (gr or 1)), C + ex
    dy, dh, y, f = (whole(g, M, C, ld, dt) for _ in range(4))
    gate = whole(g, R, C, ld, dt, -1, 2) if gr else None
    gp, gq = (torch.randint(1, 3, (C,), device=DEV, generator=g).float() for _ in range(2))
    bp, bq = ((torch.randint(-2, 3, (C,), device=DEV, generator=g).float() for _ in range(2)) if beta else (None, None))
    nm = elf.BlockNorm(C, "none", "rms", gp, bp, gq, bq, "none", gr or 1, 2.0)
    new = lambda r: torch.full((r, ld), float("nan"), dtype=DT[dt], device=DEV)[:, :C]  # noqa: E731
    vec = lambda: torch.full((C,), float("nan"), device=DEV)  # noqa: E731
    dx, df, dgate, g_post, b_post, g_pre, b_pre = new(M), new(M), new(R) if gr else None, vec(), vec(), vec(), vec()
    betas = dict(dpost_beta=b_post) if beta else {}
    elf.block_norm_bwd(nm, None, dx, dy=dy, f=f, gate=gate, df=df, dgate=dgate, dpost_gamma=g_post, **betas)
    D = dy.double()
    t = f.double() * gp + (bp if beta else 0.0)
    rows = torch.arange(M, device=DEV) // (gr or 1)
    u = 2.0 * D * (gate.double()[rows] if gr else 1.0)
    assert torch.equal(dx, dy) and torch.equal(df.double(), u * gp)
    assert torch.equal(g_post.double(), (u * f.double()).sum(0))
    if beta:
        assert torch.equal(b_post.double(), u.sum(0))
    if gr:
        want = torch.zeros((R, C), dtype=torch.float64, device=DEV).index_add_(0, rows, 2.0 * D * t)
        assert float(want.abs().max()) < 2**24
        assert torch.equal(dgate, want.float().to(DT[dt]))
    del D, t, u, rows
    # the pre norm's gradients: statistics (0, 1) make its output the stored y
    st = torch.tensor([0.0, 1.0], device=DEV).repeat(M, 1)
    betas = dict(dpre_beta=b_pre) if beta else {}
    elf.block_norm_bwd(nm, y, None, dh=dh, pre_stats=st, dpre_gamma=g_pre, **betas)
    want_g, want_b = (dh.double() * y.double()).sum(0), dh.double().sum(0)
    assert torch.equal(g_pre.double(), want_g) and (not beta or torch.equal(b_pre.double(), want_b))
    # all at once
    g2, b2 = vec(), vec()
    betas = dict(dpre_beta=b2, dpost_beta=vec()) if beta else {}
    elf.block_norm_bwd(nm, y, dx, dy=dy, dh=dh, f=f, gate=gate, df=df, dgate=dgate, pre_stats=st, dpre_gamma=g2,
                       dpost_gamma=vec(), **betas)
    assert torch.equal(g2.double(), want_g) and (not beta or torch.equal(b2.double(), want_b))
    assert ex == 0 or all(bool(torch.isnan(torch.as_strided(v, (v.shape[0], ex), (ld, 1), C).float()).all())
                          for v in (dx, df, dgate) if v is not None)


MANY = [(40_001, 128, 128, "bf16", 1, True), (40_001, 128, 128, "f16", 1, False), (10_007, 479, 481, "f16", 1, True),
        (7_001, 512, 512, "f32", 1, True), (200_003, 16, 16, "f32", 1, False), (200_003, 16, 17, "bf16", None, True),
        (9_001, 1024, 1024, "bf16", 1, False)]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_block_norm_many_rows_to_a_slot(case):
    """A gate row to each row (or none) and several rows to a slot, so that the next rows are on their way
    while one is worked on: every row's outputs against the 64-bit form."""
    M, C, ld, dt, gr, beta = case
    t, nm, act = norm_case((M, C, ld, 0, dt, "layer", "rms", "sigmoid" if gr else None, 1, 0.5, beta, 0.1))
    y, h, dx, df = (out(M, C, ld, dt) for _ in range(4))
    dg = out(M, C, ld, dt) if gr else None
    ps, qs = torch.empty((M, 2), device=DEV), torch.empty((M, 2), device=DEV)
    g = [torch.full((C,), float("nan"), device=DEV) for _ in range(4)]
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    kw = dict(dpost_beta=g[1], dpre_beta=g[3]) if beta else {}
    elf.block_norm_bwd(nm, y, dx, dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], df=df, dgate=dg, post_stats=ps,
                       pre_stats=qs, dpost_gamma=g[0], dpre_gamma=g[2], **kw)
    n = {k: np64(v) for k, v in t.items()}
    args = (n["gp"], n["bp"], n["gq"], n["bq"], act, 1, 0.5)
    ref = bp.block_norm_fwd(n["x"], n["f"], n["gate"], "layer", "rms", *args, np.float64(np.float32(0.1)), DT[dt])
    tp.check(y, ref["y"], "y")
    tp.check(h, ref["h"], "h")
    tp.check(ps, ref["post_stats"], "post_stats")
    tp.check(qs, ref["pre_stats"], "pre_stats")
    ref = bp.block_norm_bwd(n["dy"], n["dh"], np64(y), n["f"], n["gate"], "layer", "rms", *args, np64(ps), np64(qs), DT[dt])
    got = dict(dx=dx, df=df, dpost_gamma=g[0], dpre_gamma=g[2])
    got.update(dict(dpost_beta=g[1], dpre_beta=g[3]) if beta else {})
    got.update(dict(dgate=dg) if gr else {})
    for k, v in got.items():
        tp.check(v, ref[k], k)
    assert all(gap_untouched(v) for v in (y, h, dx, df, dg) if v is not None)


@pytest.mark.parametrize("gr", [1, 26])
@pytest.mark.parametrize("M,C,dt", [(9_001, 1024, "bf16"), (9_001, 640, "f16"), (3_001, 1024, "f32"), (20_011, 256, "bf16")])
def test_block_norm_outputs_together_and_one_at_a_time(M, C, dt, gr):
    """A norm without betas: its outputs have the same bits in whatever company, as long as no beta's
    gradient is asked for; and again with one (another slot for 513 to 1024 columns in 16 bits)."""
    t, nm, act = norm_case((M, C, C, 0, dt, "rms", "layer", "sigmoid", gr, 0.5, False, 0.1))
    new = lambda r=M: torch.full((r, C), float("nan"), dtype=DT[dt], device=DEV)  # noqa: E731
    vec = lambda: torch.full((C,), float("nan"), device=DEV)  # noqa: E731
    y, h, ps, qs = new(), new(), torch.empty((M, 2), device=DEV), torch.empty((M, 2), device=DEV)
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    make = dict(dx=new, df=new, dgate=lambda: new(-(-M // gr)), dpost_gamma=vec, dpre_gamma=vec)

    def run(names, **more):
        o = {k: make[k]() for k in names}
        elf.block_norm_bwd(nm, y, o.get("dx"), dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs,
                           **{k: v for k, v in o.items() if k != "dx"}, **more)
        return o

    for more in ((), ("dpre_beta",), ("dpost_beta", "dpre_beta")):
        betas = lambda: {k: vec() for k in more}  # noqa: E731
        full = run(make, **betas())
        assert all(bool(torch.isfinite(v).all()) for v in full.values())
        for k in make:
            assert torch.equal(run([k], **betas())[k], full[k]), (k, more)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,K", [(5, 300), (2_100, 300), (8_200, 300), (40, 4_200)])
def test_dense_fwd_fp4_nan_blocks_under_every_activation(M, K, act):
    """A NaN block of x or w reaches every output of its row or column, rows packed within the call and
    before it, with a residual and without."""
    N = 70
    g = torch.Generator(DEV).manual_seed(M)
    x, w = torch.randn((M, K), device=DEV, generator=g).bfloat16(), torch.randn((N, K), device=DEV, generator=g).bfloat16()
    r = torch.randn((M, N), device=DEV, generator=g).bfloat16()
    clean = elf.fp4_pack(w, elf.Fp4(N, K, DEV))
    w2, x2 = w.clone(), x.clone()
    x2[2, K - 10], x2[M - 1, 0], w2[7, 3] = float("nan"), float("-inf"), float("inf")
    w4 = elf.fp4_pack(w2, elf.Fp4(N, K, DEV))
    bad = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    bad[2], bad[M - 1], bad[:, 7] = True, True, True
    for res in (None, r):
        y, want = torch.empty((M, N), dtype=torch.bfloat16, device=DEV), torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        elf.dense_fwd_fp4(x2, w4, None, y, act=act, residual=res)
        elf.dense_fwd_fp4(x, clean, None, want, act=act, residual=res)
        assert torch.equal(torch.isnan(y), bad)
        assert torch.equal(y[~bad], want[~bad])

"""The residual block's operators on the GPU against their plain 64-bit forms (tests/block_plain.py,
which also derives the bounds), at the sizes, strides and values where they can go wrong."""
import numpy as np
import pytest
import torch

import embedding_lookup_feature_amd as elf
from tests import block_plain as bp
from tests import tower_plain as tp
from tests.test_tower_gpu import DEV, DT, gap_untouched, make_drop, np64, out, rows

pytestmark = pytest.mark.gpu


def vec(rng, n, base=0.0, scale=0.3):
    return torch.from_numpy(base + scale * rng.normal(size=n)).float().to(DEV)


def codes_of(p, fp4):
    """(codes one per value, scale bytes) of a packed array, as int64 numpy arrays."""
    c, s = (t.cpu().numpy().astype(np.int64) for t in (p.codes, p.scales))
    if fp4:
        c, s = rows_of_codes(np.stack([c & 15, c >> 4], -1)), rows_of_scales(s)
        assert (c[p.rows:] == 0).all() and (c[:, -(-p.cols // 128) * 128:] == 0).all()
        c, s = c[:p.rows], s[:p.rows, :c.shape[1] // 32]
    return c, s


def rows_of_codes(c):
    """[tiles, steps, 2, 64, 16, 2] -> [rows, columns]: lane l of fragment i holds block l / 16 of row
    8 (l % 16 / 4) + 4 i + l % 4."""
    T, S = c.shape[:2]
    return c.reshape(T, S, 2, 4, 4, 4, 32).transpose(0, 4, 2, 5, 1, 3, 6).reshape(T * 32, S * 128)


def rows_of_scales(s):
    T, S = s.shape[:2]
    return s.reshape(T, S, 2, 4, 4, 4, 4).transpose(0, 4, 2, 5, 1, 6, 3).reshape(T * 32, S * 16)


def codes_from_rows(c):
    """The inverses for whole tiles."""
    T, S = c.shape[0] // 32, c.shape[1] // 128
    return c.reshape(T, 4, 2, 4, S, 4, 32).transpose(0, 4, 2, 5, 1, 3, 6).reshape(T, S, 2, 64, 16, 2)


def scales_from_rows(s):
    T, S = s.shape[0] // 32, s.shape[1] // 16
    return s.reshape(T, 4, 2, 4, S, 4, 4).transpose(0, 4, 2, 6, 1, 3, 5).reshape(T, S, 2, 64, 4)


def new(fp4, M, K):
    p = (elf.Fp4 if fp4 else elf.Checkpoint)(M, K, DEV)
    p.codes.fill_(0xEE), p.scales.fill_(0xEE)
    return p


def check_packed(x, fp4):
    M, K = x.shape
    p = new(fp4, M, K)
    (elf.fp4_pack if fp4 else elf.ckpt_pack)(x, p)
    code, byte = codes_of(p, fp4)
    rc, rb = bp.pack(np64(x), fp4)
    assert (byte == rb).all(), (np.argwhere(byte != rb)[:3], byte[byte != rb][:3], rb[byte != rb][:3])
    if not fp4:  # either NaN of e4m3
        code = np.where((code & 127) == 127, 127, code)
    assert (code == rc).all(), (np.argwhere(code != rc)[:3], code[code != rc][:3], rc[code != rc][:3])
    return p


PACK_SIZES = [(1, 1, 1, 0), (3, 7, 9, 1), (5, 32, 32, 0), (2, 33, 40, 3), (77, 479, 480, 0), (64, 128, 136, 8),
              (13, 129, 129, 0), (300, 1024, 1024, 0), (2, 5000, 5001, 1), (1000, 4, 4, 0)]


@pytest.mark.parametrize("fp4", [False, True], ids=["8", "4"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", PACK_SIZES, ids=str)
def test_pack_is_the_definition(size, dt, fp4):
    M, K, ld, at = size
    rng = np.random.default_rng(M + K)
    x = rows(rng, M, K, ld, dt, 1.0, at=at) * torch.exp2(torch.from_numpy(rng.integers(-10, 10, size=(M, 1))).to(DEV)).to(DT[dt])
    full = torch.full((M, ld), float("nan"), dtype=DT[dt], device=DEV)
    full[:, at:at + K] = x
    check_packed(full[:, at:at + K], fp4)


@pytest.mark.parametrize("fp4", [False, True], ids=["8", "4"])
def test_pack_every_16_bit_value_against_block_maxima(fp4):
    """Every bf16 and fp16 value next to block maxima of several sizes: all ties, subnormals, both
    zeros, infinities and NaN."""
    for dt in (torch.bfloat16, torch.float16):
        all16 = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
        fin = all16[torch.isfinite(all16)]
        for top in (1.0, 1.5, 1.75, 1.7578125, 1.9921875, 448.0, 6.0, 2.0**-14, 2.0**-12):
            v = fin[fin.float().abs() <= top]
            n = -(-v.numel() // 31) * 31
            b = torch.zeros(n, dtype=dt)
            b[:v.numel()] = v
            b = torch.cat([torch.full((n // 31, 1), top, dtype=dt), b.view(-1, 31)], 1)
            check_packed(b.to(DEV), fp4)
        check_packed(all16.view(-1, 64).to(DEV), fp4)  # neighbours in size, and the non-finite ones


@pytest.mark.parametrize("fp4", [False, True], ids=["8", "4"])
def test_pack_fp32_extremes(fp4):
    rng = np.random.default_rng(7)
    e = rng.integers(-149, 128, size=(400, 1))
    x = torch.from_numpy((rng.uniform(1, 2, size=(400, 96)) * rng.choice([-1, 1], size=(400, 96)) *
                          2.0 ** np.clip(e - rng.integers(0, 14, size=(400, 96)), -149, 127))).float()
    x[0] = torch.finfo(torch.float32).max
    x[1] = torch.finfo(torch.float32).min
    x[2] = 2.0**-149
    x[3] = 0.0
    x[4] = -0.0
    x[5, 3], x[5, 40], x[6, 70], x[7] = float("inf"), float("nan"), float("-inf"), float("nan")
    check_packed(x.to(DEV), fp4)


def test_unpacking_every_code_and_scale():
    """All codes under all scale bytes, to every type (fp32 exactly, 16 bits rounded once)."""
    for fp4 in (False, True):
        n = 16 if fp4 else 256
        K = 512 if fp4 else 128
        code = np.tile(np.arange(K) % n, (508 if not fp4 else 256, 1))
        if not fp4:
            code = (code + 128 * (np.arange(code.shape[0])[:, None] % 2)) % 256
        byte = np.repeat((np.arange(code.shape[0]) % 254 + 1)[:, None], K // 32, 1)
        M = code.shape[0]
        p = new(fp4, M, K)
        raw, rs = code, byte
        if fp4:
            raw, rs = codes_from_rows(code), scales_from_rows(byte)
            raw = raw[..., 0] + 16 * raw[..., 1]
        p.codes.copy_(torch.from_numpy(np.ascontiguousarray(raw).astype(np.uint8)))
        p.scales.copy_(torch.from_numpy(np.ascontiguousarray(rs).astype(np.uint8)))
        sign = 8 if fp4 else 128
        mag = code % sign
        want = bp.values(np.where(code >= sign, mag + (8 if fp4 else 128), mag), byte, K, fp4)
        for dt in ("f32", "f16", "bf16"):
            y = torch.empty((M, K), dtype=DT[dt], device=DEV)
            elf.fp4_unpack(p, y) if fp4 else elf.ckpt_act_dropout_fwd(p, y)
            with np.errstate(over="ignore"):
                ref = torch.from_numpy(want).to(DT[dt]) if dt != "f32" else torch.from_numpy(want.astype(np.float32))
            assert torch.equal(torch.nan_to_num(y.cpu().float(), nan=-7e30), torch.nan_to_num(ref.float(), nan=-7e30)), (fp4, dt)


def test_fp4_nan_blocks():
    x = torch.ones(3, 200, device=DEV)
    x[1, 40], x[2, 199] = float("nan"), float("inf")
    p = elf.fp4_pack(x, new(True, 3, 200))
    y = elf.fp4_unpack(p, torch.empty_like(x)).cpu()
    bad = torch.zeros(3, 200, dtype=torch.bool)
    bad[1, 32:64], bad[2, 192:] = True, True
    assert torch.equal(torch.isnan(y), bad) and bool((y[~bad] == 1).all())


# ------------------------------------------------------------------------- activations from 8 bits
ACT_CASES = [
    # M, K, ld, column offset, dtype, act, p
    (1, 1, 1, 0, "f32", "gelu", 0.5), (3, 7, 8, 1, "f16", "silu", 0.1), (64, 128, 128, 0, "bf16", "relu", 0.2),
    (77, 479, 480, 0, "f16", "none", None), (33, 31, 33, 2, "f32", "silu", 0.3), (17, 257, 259, 1, "bf16", "gelu", 0.7),
    (300, 65, 65, 0, "f32", "relu", 1.0), (129, 1024, 1032, 0, "bf16", "gelu", 0.1), (50, 33, 40, 0, "f32", "none", 0.0),
    (40, 96, 96, 0, "f32", "gelu", None),
]


@pytest.mark.parametrize("case", ACT_CASES, ids=lambda c: "-".join(map(str, c)))
def test_ckpt_act_dropout(case):
    M, K, ld, at, dt, kind, p = case
    rng = np.random.default_rng(M * 1000 + K)
    x, dy = rows(rng, M, K, ld, dt, 2.0, at=at), rows(rng, M, K, ld, dt, at=at)
    y, dx = out(M, K, ld, dt, at), out(M, K, ld, dt, at)
    d, seed, offset = make_drop(p)
    ck = elf.ckpt_pack(x, new(False, M, K))
    elf.ckpt_act_dropout_fwd(ck, y, act=kind, dropout=d)
    elf.ckpt_act_dropout_bwd(dy, ck, dx, act=kind, dropout=d)
    f = tp.drop_factors(M, K, p, seed, offset) if p is not None else None
    xq = bp.rounded(np64(x), False)
    tp.check(y, tp.act_dropout_fwd(xq, kind, f, None, DT[dt]), "y")
    tp.check(dx, tp.act_dropout_bwd(np64(dy), xq, kind, f, DT[dt]), "dx")
    assert gap_untouched(y) and gap_untouched(dx)


def test_ckpt_gelu_fp32_is_accurate_in_the_tail():
    x = torch.linspace(-9.0, 3.0, 4096, device=DEV).view(-1, 32).contiguous()
    ck = elf.ckpt_pack(x, new(False, 128, 32))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    elf.ckpt_act_dropout_fwd(ck, y, act="gelu")
    elf.ckpt_act_dropout_bwd(torch.ones_like(x), ck, dx, act="gelu")
    u = torch.from_numpy(bp.rounded(np64(x), False))
    phi = 0.5 * torch.special.erfc(u * -(0.5**0.5))  # (ndtr forms 1 + erf, which is 0 from u = -8.3 down)
    # erfc's argument is rounded: its relative error grows by |u|^2 half steps of fp32, 2^-24
    tol = (16 + 4 * u.square()) * 2.0**-24
    assert bool(((y.cpu().double() - u * phi).abs() <= tol * (u * phi).abs() + 2.0**-140).all())
    pdf = torch.exp(-u * u / 2) / np.sqrt(2 * np.pi)
    assert bool(((dx.cpu().double() - phi - u * pdf).abs() <= tol * (phi + (u * pdf).abs()) + 2.0**-140).all())


def test_dropped_values_are_zero_whatever_they_held():
    M, K = 16, 64
    f = tp.drop_factors(M, K, 0.5, 9, 9)
    x = torch.full((M, K), 2.0, device=DEV)
    x[torch.from_numpy(f == 0).to(DEV)] = float("nan")
    ck = elf.ckpt_pack(x, new(False, M, K))
    y = elf.ckpt_act_dropout_fwd(ck, torch.empty_like(x), dropout=elf.Dropout(0.5, 9, 9))
    assert torch.equal(y.cpu().double(), torch.from_numpy(2.0 * f))


# ------------------------------------------------------------------------- block norm
NORM_CASES = [
    # M, C, ld, column offset, dtype, post, pre, gate, gate_rows, scale, beta, eps
    (1, 1, 1, 0, "f32", "rms", "rms", "plain", 1, 0.5, True, 0.1),
    (1, 1024, 1024, 0, "bf16", "rms", "rms", None, 1, 0.5, False, 1e-5),
    (7, 16, 16, 0, "bf16", "layer", "layer", "plain", 3, 1.0, True, 1e-5),
    (33, 24, 25, 1, "f16", "none", "rms", "sigmoid", 1, 2.0, False, 1e-5),
    (129, 40, 48, 8, "f32", "rms", "layer", "sigmoid", 129, 0.7, True, 1e-5),
    (52, 128, 128, 0, "f16", "layer", "layer", "plain", 26, 1.0, True, 1e-5),
    (70, 200, 201, 0, "bf16", "layer", "rms", "sigmoid", 7, 0.5, True, 1e-5),
    (45, 479, 480, 0, "f16", "rms", "layer", "plain", 1, 0.5, False, 1e-5),
    (300, 512, 512, 0, "bf16", "rms", "rms", "sigmoid", 1000, 1.0, False, 1e-5),
    (17, 1001, 1003, 2, "f32", "layer", "layer", None, 1, -0.5, True, 1e-5),
    (1100, 1024, 1024, 0, "bf16", "rms", "rms", "sigmoid", 1, 0.5, False, 1e-5),
    (9, 1500, 1504, 0, "f16", "layer", "rms", "sigmoid", 4, 0.5, True, 1e-5),
    (5, 4000, 4001, 1, "bf16", "rms", "layer", "plain", 2, 1.0, True, 1e-5),
    (3, 8192, 8192, 0, "f32", "layer", "layer", "sigmoid", 2, 1.0, False, 1e-5),
    (2, 16001, 16008, 0, "f16", "rms", "rms", "plain", 5, 1.0, True, 1e-5),
    (3, 32768, 32768, 0, "bf16", "layer", "layer", "sigmoid", 1, 1.0, True, 1e-5),
    (5000, 128, 128, 0, "bf16", "layer", "rms", "plain", 26, 1.0, True, 1e-5),
    (70000, 16, 16, 0, "f32", "rms", "layer", "sigmoid", 1, 1.0, True, 1e-5),
]


def norm_case(case):
    M, C, ld, at, dt, post, pre, gate, gr, scale, beta, eps = case
    rng = np.random.default_rng(M * 100 + C)
    R = -(-M // gr)
    t = dict(x=rows(rng, M, C, ld, dt, 1.0, 0.3, at), f=rows(rng, M, C, ld, dt, 2.0, 0.5, at),
             gate=rows(rng, R, C, ld, dt, 1.0, at=at) if gate else None, dy=rows(rng, M, C, ld, dt, at=at),
             dh=rows(rng, M, C, ld, dt, at=at), gp=vec(rng, C, 1.0), gq=vec(rng, C, 1.0),
             bp=vec(rng, C) if beta else None, bq=vec(rng, C) if beta else None)
    act = "sigmoid" if gate == "sigmoid" else "none"
    nm = elf.BlockNorm(C, post, pre, t["gp"], t["bp"], t["gq"], t["bq"], act, gr, scale, eps)
    return t, nm, act


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "-".join(map(str, c)))
def test_block_norm(case):
    M, C, ld, at, dt, post, pre, gate, gr, scale, beta, eps = case
    t, nm, act = norm_case(case)
    y, h, dx, df = (out(M, C, ld, dt, at) for _ in range(4))
    dgate = out(-(-M // gr), C, ld, dt, at) if gate else None
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    ps, qs = nan(M, 2) if post != "none" else None, nan(M, 2)
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    s = np.float64(np.float32(scale))
    e = np.float64(np.float32(eps))
    n = {k: np64(v) for k, v in t.items()}
    ref = bp.block_norm_fwd(n["x"], n["f"], n["gate"], post, pre, n["gp"], n["bp"], n["gq"], n["bq"], act, gr, s, e, DT[dt])
    tp.check(y, ref["y"], "y")
    tp.check(h, ref["h"], "h")
    tp.check(qs, ref["pre_stats"], "pre_stats")
    if ps is not None:
        tp.check(ps, ref["post_stats"], "post_stats")
    g = [nan(C) for _ in range(4)]
    elf.block_norm_bwd(nm, y, dx, dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], df=df, dgate=dgate, post_stats=ps,
                       pre_stats=qs, dpost_gamma=g[0], dpost_beta=g[1], dpre_gamma=g[2], dpre_beta=g[3])
    ref = bp.block_norm_bwd(n["dy"], n["dh"], np64(y), n["f"], n["gate"], post, pre, n["gp"], n["bp"], n["gq"], n["bq"], act,
                            gr, s, np64(ps), np64(qs), DT[dt])
    for k, v in (("dx", dx), ("df", df), ("dgate", dgate), ("dpost_gamma", g[0]), ("dpost_beta", g[1]), ("dpre_gamma", g[2]),
                 ("dpre_beta", g[3])):
        if v is not None:
            tp.check(v, ref[k], k)
    assert all(gap_untouched(v) for v in (y, h, dx, df, dgate) if v is not None)


@pytest.mark.parametrize("C,dt", [(16, "f32"), (479, "bf16"), (1024, "f16"), (2048, "bf16")])
def test_block_norm_parts(C, dt):
    """Outputs and operands left out: a plain norm, the last block's sum, a gate without a residual."""
    M = 37
    t, nm, act = norm_case((M, C, C, 0, dt, "layer", "rms", "sigmoid", 5, 0.5, True, 1e-5))
    full = {k: torch.empty((M, C), dtype=DT[dt], device=DEV) for k in ("y", "h", "dx", "df")}
    ps, qs = torch.empty((M, 2), device=DEV), torch.empty((M, 2), device=DEV)
    E = lambda r=M: torch.full((r, C), float("nan"), dtype=DT[dt], device=DEV)  # noqa: E731
    elf.block_norm_fwd(nm, t["x"], full["y"], full["h"], f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    y, h = E(), E()
    elf.block_norm_fwd(nm, t["x"], y, None, f=t["f"], gate=t["gate"])
    elf.block_norm_fwd(nm, t["x"], None, h, f=t["f"], gate=t["gate"])
    assert torch.equal(y, full["y"]) and torch.equal(h, full["h"])
    zero = torch.zeros_like(t["x"])
    a, b = E(), E()
    elf.block_norm_fwd(nm, None, a, None, f=t["f"], gate=t["gate"])
    elf.block_norm_fwd(nm, zero, b, None, f=t["f"], gate=t["gate"])
    assert torch.equal(a, b)
    # h alone: the norm of x, and its gradient
    n = {k: np64(v) for k, v in t.items()}
    e = np.float64(np.float32(1e-5))
    q2 = torch.empty((M, 2), device=DEV)
    elf.block_norm_fwd(nm, t["x"], None, h, pre_stats=q2)
    ref = bp.block_norm_fwd(n["x"], None, None, "layer", "rms", n["gp"], n["bp"], n["gq"], n["bq"], act, 5, 0.5, e, DT[dt])
    tp.check(h, ref["h"], "h")
    dx = E()
    dg = torch.empty(C, device=DEV)
    elf.block_norm_bwd(nm, t["x"], dx, dh=t["dh"], pre_stats=q2, dpre_gamma=dg)
    ref = bp.block_norm_bwd(None, n["dh"], n["x"], None, None, "layer", "rms", n["gp"], n["bp"], n["gq"], n["bq"], act, 5, 0.5,
                            None, np64(q2), DT[dt])
    tp.check(dx, ref["dx"], "dx")
    tp.check(dg, ref["dpre_gamma"], "dpre_gamma")
    # the last block: dy alone; every other output may be left out
    df, dgt = E(), E(8)
    elf.block_norm_bwd(nm, None, None, dy=t["dy"], f=t["f"], gate=t["gate"], df=df, dgate=dgt, post_stats=ps)
    ref = bp.block_norm_bwd(n["dy"], None, None, n["f"], n["gate"], "layer", "rms", n["gp"], n["bp"], n["gq"], n["bq"], act, 5,
                            0.5, np64(ps), None, DT[dt])
    tp.check(df, ref["df"], "df")
    tp.check(dgt, ref["dgate"], "dgate")
    # all at once and one at a time give the same bits
    g = {k: torch.empty(C, device=DEV) for k in ("dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")}
    kw = dict(dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    elf.block_norm_bwd(nm, full["y"], full["dx"], df=full["df"], **g, **kw)
    dx = E()
    elf.block_norm_bwd(nm, full["y"], dx, **kw)
    assert torch.equal(dx, full["dx"])
    for k in g:
        one = torch.full((C,), float("nan"), device=DEV)
        elf.block_norm_bwd(nm, full["y"], None, **{k: one}, **kw)
        assert torch.equal(one, g[k]), k


def test_block_norm_empty_batch():
    nm = elf.BlockNorm(8, "rms", "rms")
    e = torch.empty((0, 8), device=DEV)
    st = torch.empty((0, 2), device=DEV)
    g = torch.full((8,), float("nan"), device=DEV)
    elf.block_norm_fwd(nm, e, e.clone(), e.clone(), f=e)
    elf.block_norm_bwd(nm, e, e.clone(), dy=e, dh=e, f=e, df=e.clone(), post_stats=st, pre_stats=st, dpre_gamma=g)
    assert bool((g == 0).all())


def test_block_norm_constant_rows_and_far_means():
    """A constant row (variance 0) and rows far from zero: centred before they are scaled."""
    M, C = 12, 320
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(M, C)) + 1000.0 * np.arange(M)[:, None]).float().to(DEV)
    x[0] = 7.0
    nm = elf.BlockNorm(C, pre="layer")
    h, st = torch.empty_like(x), torch.empty((M, 2), device=DEV)
    elf.block_norm_fwd(nm, x, None, h, pre_stats=st)
    ref = bp.block_norm_fwd(np64(x), None, None, "none", "layer", None, None, None, None, "none", 1, 1.0,
                            np.float64(np.float32(1e-5)), torch.float32)
    tp.check(h, ref["h"], "h")
    tp.check(st, ref["pre_stats"], "stats")


def test_block_norm_nan_rows_stay_in_their_rows():
    M, C = 40, 96
    t, nm, act = norm_case((M, C, C, 0, "f32", "rms", "layer", "plain", 1, 0.5, True, 1e-5))
    t["f"][3, 5], t["x"][9, 0], t["gate"][20, 7] = float("nan"), float("inf"), float("nan")
    y, h = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"])
    bad = torch.isnan(h).any(1).cpu().numpy()
    assert set(np.flatnonzero(bad)) == {3, 9, 20} and set(np.flatnonzero(~torch.isfinite(y).all(1).cpu().numpy())) == {3, 9, 20}


# ------------------------------------------------------------------------- dense backward from 8 bits
DENSE_BWD = [
    # M, K, N, extra columns, dtype, act, p, residual, dx?
    (1, 1, 1, 0, "bf16", "relu", None, False, True), (5, 7, 3, 1, "f16", "gelu", 0.5, True, True),
    (33, 32, 16, 0, "bf16", "silu", 0.1, True, True), (130, 96, 72, 8, "f16", "none", None, False, True),
    (257, 479, 129, 1, "bf16", "gelu", 0.2, True, True), (300, 100, 40, 0, "bf16", "relu", None, False, False),
    (700, 33, 520, 0, "f16", "silu", None, True, True), (24_600, 1_000, 1_032, 0, "bf16", "silu", 0.3, True, True),
    (5_000, 1_032, 1_032, 0, "f16", "gelu", 0.3, True, True), (4_200, 1_031, 136, 0, "bf16", "silu", 0.3, False, True),
    (5_700, 520, 1_032, 0, "bf16", "silu", 0.3, False, True), (33_000, 264, 72, 0, "f16", "gelu", 0.3, True, True),
    (2_048, 64, 64, 0, "bf16", "gelu", None, False, True), (4099, 479, 256, 1, "f16", "silu", 0.2, False, True),
]


@pytest.mark.parametrize("case", DENSE_BWD, ids=lambda c: "-".join(map(str, c)))
def test_dense_bwd_ckpt(case):
    M, K, N, ex, dt, kind, p, res, want_dx = case
    rng = np.random.default_rng(M + K + N)
    x, pre = rows(rng, M, K, K, dt, 1.0), rows(rng, M, K, K + ex, dt, 1.5)
    w = rows(rng, N, K, K, dt, 1 / np.sqrt(N)).contiguous()
    dz = rows(rng, M, N, N + ex, dt)
    dres = rows(rng, M, K, K + ex, dt) if res else None
    xq, pq = elf.ckpt_pack(x, new(False, M, K)), elf.ckpt_pack(pre, new(False, M, K))
    dx, dzb = (out(M, K, K + ex, dt), out(M, K, K + ex, dt)) if want_dx else (None, None)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    dw, db = nan(N, K), nan(N)
    d, seed, offset = make_drop(p)
    elf.dense_bwd_ckpt(xq, w, dz, dw, db, dx=dx, dres=dres, dzb=dzb, pre=pq if kind != "none" else None, act=kind, dropout=d)
    f = tp.drop_factors(M, K, p, seed, offset) if p is not None else None
    x8, p8 = bp.rounded(np64(x), False), bp.rounded(np64(pre), False)
    ref = tp.dense_bwd(x8, np64(w), np64(dz), np64(dres), p8 if kind != "none" else None, kind, f, DT[dt])
    tp.check(dw, ref["dw"], "dw")
    tp.check(db, ref["db"], "db")
    if want_dx:
        tp.check(dx, ref["dx"], "dx")
        tp.check(dzb, ref["dzb"], "dzb")
        assert gap_untouched(dx) and gap_untouched(dzb)
    dw2 = nan(N, K)
    elf.dense_bwd_ckpt(xq, w, dz, dw2, dx=out(M, K, K, dt) if want_dx else None)
    assert torch.equal(dw, dw2)


def test_dense_bwd_ckpt_empty_batch():
    K, N = 24, 40
    z = lambda m, n: torch.empty((m, n), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dw, db = torch.ones((N, K), device=DEV), torch.ones(N, device=DEV)
    elf.dense_bwd_ckpt(elf.Checkpoint(0, K, DEV), z(N, K), z(0, N), dw, db, dx=z(0, K))
    assert bool((dw == 0).all()) and bool((db == 0).all())


# ------------------------------------------------------------------------- dense layer in 4 bits
DENSE_FP4 = [
    # M, K, N, extra columns, dtype, act, residual, bias
    (1, 1, 1, 0, "bf16", "none", False, True), (1, 1024, 1024, 0, "bf16", "gelu", True, True),
    (3, 129, 17, 1, "f16", "silu", True, True), (16, 512, 64, 0, "bf16", "relu", False, False),
    (17, 479, 1001, 1, "f16", "relu", False, True), (77, 512, 1024, 0, "f16", "silu", False, True),
    (257, 100, 130, 8, "bf16", "gelu", True, True), (300, 2048, 512, 0, "bf16", "none", True, False),
    (4099, 479, 1001, 1, "f16", "relu", False, True), (9000, 256, 264, 0, "bf16", "gelu", True, True),
    (33_000, 40, 264, 0, "bf16", "silu", True, True), (2, 5000, 33, 0, "f16", "none", False, True),
    (40_000, 24, 1, 0, "bf16", "none", False, True), (64, 4096, 2048, 0, "bf16", "gelu", False, True),
    (9_000, 4096, 520, 0, "bf16", "none", False, True), (8_300, 8_200, 520, 0, "bf16", "silu", True, True),
    (8_200, 8_201, 515, 1, "f16", "none", False, False), (37, 70_000, 100, 0, "bf16", "none", True, True),
]


@pytest.mark.parametrize("case", DENSE_FP4, ids=lambda c: "-".join(map(str, c)))
def test_dense_fwd_fp4(case):
    M, K, N, ex, dt, kind, res, bias = case
    rng = np.random.default_rng(M + K + N)
    x, w = rows(rng, M, K, K + ex, dt, 1.0), rows(rng, N, K, K, dt, 1 / np.sqrt(K))
    b = vec(rng, N) if bias else None
    r = rows(rng, M, N, N + ex, dt) if res else None
    y = out(M, N, N + ex, dt)
    w4 = elf.fp4_pack(w, new(True, N, K))
    elf.dense_fwd_fp4(x, w4, b, y, act=kind, residual=r)
    ref = bp.dense_fp4(bp.rounded(np64(x), True), bp.rounded(np64(w), True), np64(b), kind, np64(r), DT[dt])
    tp.check(y, ref, "y")
    assert gap_untouched(y)


@pytest.mark.parametrize("M", [5, 300])
def test_dense_fwd_fp4_nan_blocks(M):
    K, N = 300, 70
    rng = np.random.default_rng(4)
    x, w = rows(rng, M, K, K, "bf16").contiguous(), rows(rng, N, K, K, "bf16").contiguous()
    x[2, 290], w[7, 3] = float("nan"), float("inf")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    elf.dense_fwd_fp4(x, elf.fp4_pack(w, new(True, N, K)), None, y)
    bad = torch.zeros((M, N), dtype=torch.bool)
    bad[2], bad[:, 7] = True, True
    assert torch.equal(torch.isnan(y).cpu(), bad)


# ------------------------------------------------------------------------- streams, graphs, offsets
def chain(t, nm, ws):
    """A residual block as it is trained and served, every operator once; its outputs by name."""
    M, C = t["x"].shape
    E = lambda dt=t["x"].dtype, *s: torch.full(s or (M, C), float("nan"), dtype=dt, device=DEV)  # noqa: E731
    f32 = torch.float32
    o = dict(y=E(), h=E(), ps=E(f32, M, 2), qs=E(f32, M, 2), z=E(), a=E(), da=E(), dh=E(), dw=E(f32, C, C), db=E(f32, C),
             dx=E(), df=E(), dg=E(), gp=E(f32, C), gq=E(f32, C), s=E())
    hq, zq, w4 = elf.Checkpoint(M, C, DEV), elf.Checkpoint(M, C, DEV), elf.Fp4(C, C, DEV)

    def go(stream=None):
        kw = dict(stream=stream)
        elf.block_norm_fwd(nm, t["x"], o["y"], o["h"], f=t["f"], gate=t["gate"], post_stats=o["ps"], pre_stats=o["qs"], **kw)
        elf.ckpt_pack(o["h"], hq, **kw)
        elf.dense_fwd(o["h"], t["w"], None, o["z"], **kw)
        elf.ckpt_pack(o["z"], zq, **kw)
        elf.ckpt_act_dropout_fwd(zq, o["a"], act="gelu", **kw)
        elf.ckpt_act_dropout_bwd(t["dy"], zq, o["da"], act="gelu", **kw)
        elf.dense_bwd_ckpt(hq, t["w"], o["da"], o["dw"], o["db"], dx=o["dh"], workspace=ws, **kw)
        elf.block_norm_bwd(nm, o["y"], o["dx"], dy=t["dy"], dh=o["dh"], f=t["f"], gate=t["gate"], df=o["df"], dgate=o["dg"],
                           post_stats=o["ps"], pre_stats=o["qs"], dpost_gamma=o["gp"], dpre_gamma=o["gq"], workspace=ws, **kw)
        elf.fp4_pack(t["w"], w4, **kw)
        elf.dense_fwd_fp4(o["h"], w4, None, o["s"], act="gelu", residual=o["y"], workspace=ws, **kw)

    return go, o


def block(M=700, C=160):
    t, nm, act = norm_case((M, C, C, 0, "bf16", "rms", "layer", "sigmoid", 1, 0.5, False, 1e-5))
    t = {k: v.contiguous() if v is not None else None for k, v in t.items()}
    t["w"] = (torch.randn(C, C, device=DEV, generator=torch.Generator(DEV).manual_seed(1)) / C**0.5).bfloat16()
    ws = torch.empty(max(elf.dense_bwd_ckpt_workspace_bytes(M, C, C), elf.block_norm_bwd_workspace_bytes(nm, M),
                         elf.dense_fwd_fp4_workspace_bytes(M, C, C)), dtype=torch.uint8, device=DEV)
    return t, nm, ws


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def test_calls_follow_the_given_stream_and_the_current_one():
    t, nm, ws = block()
    go, want = chain(t, nm, ws)
    go()
    assert all(bool(torch.isfinite(v).all()) for v in want.values())
    side = torch.cuda.Stream()
    for how in ("given", "handle", "current"):
        go, got = chain(t, nm, None)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side) if how == "current" else torch.cuda.stream(None):
            go(**({"stream": side} if how == "given" else {"stream": side.cuda_stream} if how == "handle" else {}))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert same(want, got), how


def test_a_captured_block_replays():
    t, nm, ws = block(130, 64)
    go, o = chain(t, nm, ws)
    go()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go()
    ws2 = torch.empty_like(ws)
    for k in range(4):
        t["f"].copy_(torch.randn(t["f"].shape, device=DEV, generator=torch.Generator(DEV).manual_seed(k)))
        for v in o.values():
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager, e = chain(t, nm, ws2)
        eager()
        torch.cuda.synchronize()
        assert same(o, e), k


def test_two_streams_at_once():
    t, nm, ws = block()
    go, want = chain(t, nm, ws)
    go()
    torch.cuda.synchronize()
    runs = [chain(t, nm, torch.empty_like(ws)) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in runs]
    for (r, _), s in zip(runs, streams):
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            r(stream=s)
    torch.cuda.synchronize()
    assert all(same(want, o) for _, o in runs)


def test_rows_past_32_bit_offsets():
    """Row strides of 2^20 elements: the last rows of 2300 lie past 2^32 bytes."""
    M, C, ld = 2_300, 64, 1 << 20
    big = torch.empty((M, ld), dtype=torch.bfloat16, device=DEV)
    at = iter(range(0, 64 * 128, 128))
    far = lambda src=None: (lambda v: v if src is None else v.copy_(src))(big[:, (a := next(at)):a + C])  # noqa: E731
    t, nm, act = norm_case((M, C, C, 0, "bf16", "rms", "layer", "sigmoid", 1, 0.5, True, 1e-5))
    st = [torch.empty((M, 2), device=DEV) for _ in range(4)]
    near = [torch.empty((M, C), dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    elf.block_norm_fwd(nm, t["x"], near[0], near[1], f=t["f"], gate=t["gate"], post_stats=st[0], pre_stats=st[1])
    y, h = far(), far()
    elf.block_norm_fwd(nm, far(t["x"]), y, h, f=far(t["f"]), gate=far(t["gate"]), post_stats=st[2], pre_stats=st[3])
    assert torch.equal(y, near[0]) and torch.equal(h, near[1]) and torch.equal(st[1], st[3])
    kw = dict(post_stats=st[0], pre_stats=st[1])
    elf.block_norm_bwd(nm, near[0], near[2], dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], df=near[3], dgate=near[4], **kw)
    dx, df, dg = far(), far(), far()
    elf.block_norm_bwd(nm, y, dx, dy=far(t["dy"]), dh=far(t["dh"]), f=far(t["f"]), gate=far(t["gate"]), df=df, dgate=dg, **kw)
    assert torch.equal(dx, near[2]) and torch.equal(df, near[3]) and torch.equal(dg, near[4])
    a, b = elf.ckpt_pack(t["x"], new(False, M, C)), elf.ckpt_pack(far(t["x"]), new(False, M, C))
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    v = far()
    elf.ckpt_act_dropout_fwd(a, near[5], act="gelu")
    elf.ckpt_act_dropout_fwd(a, v, act="gelu")
    assert torch.equal(v, near[5])
    w4 = elf.fp4_pack(t["f"][:72].contiguous(), new(True, 72, C))
    s, sf = torch.empty((M, 72), dtype=torch.bfloat16, device=DEV), big[:, 20_000:20_072]
    elf.dense_fwd_fp4(t["x"], w4, None, s)
    elf.dense_fwd_fp4(far(t["x"]), w4, None, sf)
    assert torch.equal(s, sf)


def test_packed_arrays_past_32_bit_offsets():
    """4.3e9 columns: the codes of the last rows lie past 2^32 bytes."""
    M, K = 4_200, 1 << 20
    x = torch.randn((1, K), device=DEV, generator=torch.Generator(DEV).manual_seed(3)).bfloat16().expand(M, K)
    p = elf.Checkpoint(M, K, DEV)
    elf.ckpt_pack(x.contiguous(), p)
    assert torch.equal(p.codes[0], p.codes[-1]) and torch.equal(p.scales[0], p.scales[-1])
    y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    elf.ckpt_act_dropout_fwd(p, y)
    assert torch.equal(y[0], y[-1])
    ref = torch.from_numpy(bp.rounded(np64(x[:1, :4096].contiguous()), False))
    assert torch.equal(y[-1:, :4096].cpu().double(), ref)


# ------------------------------------------------------------------------- more of the block norm
@pytest.mark.parametrize("M,C,ld,gr,dt", [
    (70_001, 16, 16, 26, "f32"),      # runs of one row and fewer
    (70_000, 24, 25, 26, "bf16"),     # rows at odd addresses
    (30_000, 128, 128, 29_999, "f16"),  # two gate rows, each in thousands of slots
    (40_000, 64, 64, 40_000, "f32"),  # one gate row
    (2_000, 1024, 1024, 7, "bf16"), (1_500, 1024, 1025, 100, "f16"), (700, 2048, 2048, 3, "f32"),
    (900, 4096, 4096, 50, "bf16"), (300, 8200, 8200, 11, "f16"), (100_003, 8, 8, 2, "bf16"),
])
def test_block_norm_shared_gates(M, C, ld, gr, dt):
    """Gate rows inside a slot's run of rows, across two and across very many; the last one cut."""
    t, nm, act = norm_case((M, C, ld, 0, dt, "rms", "layer", "sigmoid", gr, 0.5, True, 0.1))
    R = -(-M // gr)
    y, h, dx, df, dg = out(M, C, ld, dt), out(M, C, ld, dt), out(M, C, ld, dt), out(M, C, ld, dt), out(R, C, ld, dt)
    ps, qs = torch.empty((M, 2), device=DEV), torch.empty((M, 2), device=DEV)
    g = [torch.full((C,), float("nan"), device=DEV) for _ in range(4)]
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    elf.block_norm_bwd(nm, y, dx, dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], df=df, dgate=dg, post_stats=ps,
                       pre_stats=qs, dpost_gamma=g[0], dpost_beta=g[1], dpre_gamma=g[2], dpre_beta=g[3])
    n = {k: np64(v) for k, v in t.items()}
    eps = np.float64(np.float32(0.1))
    ref = bp.block_norm_fwd(n["x"], n["f"], n["gate"], "rms", "layer", n["gp"], n["bp"], n["gq"], n["bq"], act, gr, 0.5, eps, DT[dt])
    tp.check(y, ref["y"], "y")
    tp.check(h, ref["h"], "h")
    ref = bp.block_norm_bwd(n["dy"], n["dh"], np64(y), n["f"], n["gate"], "rms", "layer", n["gp"], n["bp"], n["gq"], n["bq"],
                            act, gr, 0.5, np64(ps), np64(qs), DT[dt])
    for k, v in (("dx", dx), ("df", df), ("dgate", dg), ("dpost_gamma", g[0]), ("dpost_beta", g[1]), ("dpre_gamma", g[2]),
                 ("dpre_beta", g[3])):
        tp.check(v, ref[k], k)
    assert all(gap_untouched(v) for v in (y, h, dx, df, dg))
    dg2 = out(R, C, ld, dt)
    elf.block_norm_bwd(nm, y, None, dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], dgate=dg2, post_stats=ps, pre_stats=qs)
    assert torch.equal(dg, dg2)


def test_block_norm_aligned_and_loose_rows_agree():
    """The same rows at aligned and at odd addresses: the same sums in the same order, the same bits."""
    M, C = 333, 256
    t, nm, act = norm_case((M, C, C, 0, "bf16", "layer", "rms", "plain", 5, 0.5, True, 1e-5))
    got = []
    for ld, at in ((C, 0), (C + 3, 1)):
        v = {k: (lambda o: o.copy_(s))(out(s.shape[0], C, ld, "bf16", at)) if s is not None and s.dim() == 2 else s for k, s in t.items()}
        y, h, dx, df, dg = (out(r, C, ld, "bf16", at) for r in (M, M, M, M, -(-M // 5)))
        ps, qs = torch.empty((M, 2), device=DEV), torch.empty((M, 2), device=DEV)
        g = [torch.empty(C, device=DEV) for _ in range(4)]
        elf.block_norm_fwd(nm, v["x"], y, h, f=v["f"], gate=v["gate"], post_stats=ps, pre_stats=qs)
        elf.block_norm_bwd(nm, y, dx, dy=v["dy"], dh=v["dh"], f=v["f"], gate=v["gate"], df=df, dgate=dg, post_stats=ps,
                           pre_stats=qs, dpost_gamma=g[0], dpost_beta=g[1], dpre_gamma=g[2], dpre_beta=g[3])
        got.append([y, h, dx, df, dg, ps, qs, *g])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_block_norm_gradients_against_differences():
    """fp32 gradients along random directions against differences of the plain 64-bit forward."""
    M, C, gr, s = 12, 40, 4, 0.5
    t, nm, act = norm_case((M, C, C, 0, "f32", "layer", "rms", "sigmoid", gr, s, True, 1e-3))
    E = lambda *z: torch.empty(z, device=DEV)  # noqa: E731
    y, h, dx, df, dg, ps, qs = E(M, C), E(M, C), E(M, C), E(M, C), E(3, C), E(M, 2), E(M, 2)
    g = [E(C) for _ in range(4)]
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    elf.block_norm_bwd(nm, y, dx, dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], df=df, dgate=dg, post_stats=ps,
                       pre_stats=qs, dpost_gamma=g[0], dpost_beta=g[1], dpre_gamma=g[2], dpre_beta=g[3])
    v = {k: np64(a) for k, a in t.items()}

    def loss(**k):
        w = {**v, **k}
        o = bp.block_norm_fwd(w["x"], w["f"], w["gate"], "layer", "rms", w["gp"], w["bp"], w["gq"], w["bq"], act, gr, s, 1e-3,
                              torch.float32)
        return float((o["y"][0] * v["dy"]).sum() + (o["h"][0] * v["dh"]).sum())

    rng = np.random.default_rng(8)
    for k, grad in (("x", dx), ("f", df), ("gate", dg), ("gp", g[0]), ("bp", g[1]), ("gq", g[2]), ("bq", g[3])):
        d = rng.normal(size=v[k].shape)
        step = 1e-5
        diff = (loss(**{k: v[k] + step * d}) - loss(**{k: v[k] - step * d})) / (2 * step)
        # differences are off by the third derivative times 1e-10; the gradients by some 1e3 fp32 steps
        assert abs((np64(grad) * d).sum() - diff) <= 1e-4 * np.abs(np64(grad) * d).sum(), k


# ------------------------------------------------------------------------- more of the dense layer in 4 bits
@pytest.mark.parametrize("M,K,N,dt", [
    (9, 18_000, 40, "bf16"), (9_001, 9_700, 264, "f16"), (33_000, 4_900, 136, "bf16"), (33_001, 4_700, 24, "f16"),
    (70_001, 96, 40, "bf16"), (8_192, 520, 1_032, "bf16"), (20_000, 8, 8, "f16"), (20_000, 7, 300, "bf16"), (500, 300, 7, "bf16"),
])
def test_dense_fwd_fp4_forms(M, K, N, dt):
    """Rows packed before the product and within it, 16, 32 and 64 a workgroup, narrow sizes: against
    64-bit products of the unpacked operands (packing is tested on its own)."""
    g = torch.Generator(DEV).manual_seed(M)
    x = torch.randn((M, K + 1), device=DEV, generator=g).to(DT[dt])[:, 1:]
    w = (torch.randn((N, K), device=DEV, generator=g) / K**0.5).to(DT[dt])
    b, r = torch.randn(N, device=DEV, generator=g), torch.randn((M, N), device=DEV, generator=g).to(DT[dt])
    y = out(M, N, N + 3, dt, 2)
    w4 = elf.fp4_pack(w, new(True, N, K))
    elf.dense_fwd_fp4(x, w4, b, y, act="silu", residual=r)
    xv = elf.fp4_unpack(elf.fp4_pack(x, new(True, M, K)), torch.empty((M, K), device=DEV))
    wv = elf.fp4_unpack(w4, torch.empty((N, K), device=DEV))
    wd = wv.double().t().contiguous()
    for a in range(0, M, 4096):
        e = min(M, a + 4096)
        z = xv[a:e].double() @ wd + b.double()
        s = xv[a:e].double().abs() @ wd.abs() + b.double().abs()
        act = z * torch.sigmoid(z)
        ref = act + r[a:e].double()
        tol = 1.13 * 2 * (-(-K // 128) * 128 + 2) * 2.0**-24 * s + z.abs() * 2.0**-20 + 4 * 2.0**-24 * (act.abs() + ref.abs())
        tol = tol + ref.abs() * torch.finfo(DT[dt]).eps / 2 * (1 + 2 * torch.finfo(DT[dt]).eps) + torch.finfo(DT[dt]).smallest_normal * torch.finfo(DT[dt]).eps / 2
        assert bool(((y[a:e].double() - ref).abs() <= tol).all()), a
    assert gap_untouched(y)


def test_a_call_on_another_devices_tensors_is_refused_or_follows_them():
    """One device here: operands on the host next to device ones are refused by name."""
    M, C = 4, 32
    x = torch.randn(M, C, device=DEV)
    nm = elf.BlockNorm(C)
    with pytest.raises(ValueError, match="h must be"):
        elf.block_norm_fwd(nm, x, None, torch.empty(M, C))
    with pytest.raises(ValueError, match="y must be"):
        elf.ckpt_act_dropout_fwd(elf.Checkpoint(M, C, DEV), torch.empty(M, C))
    with pytest.raises(ValueError, match="ckpt must be"):
        elf.ckpt_pack(x, elf.Checkpoint(M, C + 1, DEV))
    with pytest.raises(ValueError, match="packed must be"):
        elf.fp4_pack(x, elf.Checkpoint(M, C, DEV))
    with pytest.raises(ValueError, match="workspace"):
        elf.block_norm_bwd(nm, x, torch.empty_like(x), dh=x, pre_stats=torch.empty((M, 2), device=DEV), workspace=torch.empty(64))


# ------------------------------------------------------------------------- workspaces of the binding's own
def own_workspace_calls(stream):
    r = lambda *s: torch.randn(*s, device=DEV, generator=torch.Generator(DEV).manual_seed(sum(s))).bfloat16()  # noqa: E731
    M, C, K, N = 5_000, 256, 250, 264
    nm = elf.BlockNorm(C, "rms", "layer", gate_rows=7)
    x, dy, f, gate = r(M, C), r(M, C).flip(0).contiguous(), r(M, C) * 2, r(-(-M // 7), C)
    st = [torch.rand((M, 2), device=DEV, generator=torch.Generator(DEV).manual_seed(k)) for k in range(2)]
    norm = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate), *(torch.empty(C, device=DEV) for _ in range(4))]
    x8 = elf.ckpt_pack(r(M, K), elf.Checkpoint(M, K, DEV))
    w, dz = r(N, K), r(M, N)
    dense = [torch.empty((M, K), dtype=torch.bfloat16, device=DEV), torch.empty((N, K), device=DEV), torch.empty(N, device=DEV)]
    wide = r(8_200, 9_600)
    w4, y = elf.fp4_pack(r(24, 9_600), elf.Fp4(24, 9_600, DEV)), torch.empty((8_200, 24), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    return {
        "block_norm_bwd": (lambda: elf.block_norm_bwd(nm, x, norm[0], dy=dy, dh=dy, f=f, gate=gate, df=norm[1], dgate=norm[2],
                                                      post_stats=st[0], pre_stats=st[1], dpost_gamma=norm[3], dpost_beta=norm[4],
                                                      dpre_gamma=norm[5], dpre_beta=norm[6], stream=stream),
                           norm, elf.block_norm_bwd_workspace_bytes(nm, M)),
        "dense_bwd_ckpt": (lambda: elf.dense_bwd_ckpt(x8, w, dz, dense[1], dense[2], dx=dense[0], stream=stream), dense,
                           elf.dense_bwd_ckpt_workspace_bytes(M, K, N)),
        "dense_fwd_fp4": (lambda: elf.dense_fwd_fp4(wide, w4, None, y, stream=stream), [y],
                          elf.dense_fwd_fp4_workspace_bytes(8_200, 9_600, 24)),
    }


@pytest.mark.parametrize("name", ["block_norm_bwd", "dense_bwd_ckpt", "dense_fwd_fp4"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_current_streams_allocations_do_not_reach_the_workspace(name, handle):
    side = torch.cuda.Stream()
    call, outs, need = own_workspace_calls(None)[name]
    assert need > 0, "the case needs a workspace"
    call()
    want = [t.clone() for t in outs]
    call, outs, need = own_workspace_calls(side.cuda_stream if handle else side)[name]
    filler = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # work of some milliseconds in front of the call
        for _ in range(40):
            filler.fill_(1)
    call()
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255) for n in (need, need, need // 2 + 512)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    assert all(bool((t == 255).all()) for t in junk)


def test_dense_fwd_fp4_packed_rows_end_in_half_a_workgroup():
    """Rows packed first, an odd number of tiles of 32 rows, 64 rows a workgroup: the tile behind the
    last is not read (the workspace ends with the last)."""
    M, K, N = 8_200, 4_200, 24
    g = torch.Generator(DEV).manual_seed(1)
    x, w = torch.randn((M, K), device=DEV, generator=g).bfloat16(), torch.randn((N, K), device=DEV, generator=g).bfloat16()
    w4, need = elf.fp4_pack(w, new(True, N, K)), elf.dense_fwd_fp4_workspace_bytes(M, K, N)
    room = torch.full((need + 65_536,), 0xFF, dtype=torch.uint8, device=DEV)
    y, cut = out(M, N, N, "bf16"), out(8, N, N, "bf16")
    elf.dense_fwd_fp4(x, w4, None, y, workspace=room[:need])
    elf.dense_fwd_fp4(x[-8:], w4, None, cut)
    assert torch.equal(y[-8:], cut) and bool((room[need:] == 0xFF).all())


def test_an_infinite_gate_reaches_its_own_rows_only():
    """Slots with one row less than their workgroup's first take a step without a row: their last
    gate row, here infinite, must not meet its zeros."""
    M, C = 2_050, 1024
    ones = torch.ones((M, C), device=DEV)
    gate = torch.ones((M // 2, C), device=DEV)
    gate[2, 5] = float("inf")  # rows 4 and 5, the third and the fourth slot's only ones
    nm = elf.BlockNorm(C, post="none", pre="rms", gate_rows=2)
    dgamma = torch.empty(C, device=DEV)
    elf.block_norm_bwd(nm, None, None, dy=ones, f=ones, gate=gate, dpost_gamma=dgamma)
    assert bool(dgamma[5].isposinf()) and bool((torch.cat([dgamma[:5], dgamma[6:]]) == M).all())


@pytest.mark.parametrize("M,C,ex,beta,gr", [
    (3_001, 1000, 0, False, 1), (3_001, 1000, 0, True, 1), (3_001, 1000, 1, True, 7), (2_500, 600, 0, True, 300),
    (1_700, 4000, 0, True, 1), (1_700, 4000, 8, False, 5), (1_300, 3001, 1, True, 3), (600, 8192, 0, False, 1),
    (600, 8000, 8, True, 9),
])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_block_norm_rows_of_several_wavefronts(M, C, ex, beta, gr, dt):
    """Two, eight and sixteen wavefronts a row, one and two rows a workgroup, with betas and without."""
    t, nm, act = norm_case((M, C, C + ex, 0, dt, "layer", "layer", "sigmoid", gr, 0.5, beta, 1e-5))
    R = -(-M // gr)
    y, h, dx, df, dg = out(M, C, C + ex, dt), out(M, C, C + ex, dt), out(M, C, C + ex, dt), out(M, C, C + ex, dt), out(R, C, C + ex, dt)
    ps, qs = torch.empty((M, 2), device=DEV), torch.empty((M, 2), device=DEV)
    g = [torch.full((C,), float("nan"), device=DEV) for _ in range(4)]
    elf.block_norm_fwd(nm, t["x"], y, h, f=t["f"], gate=t["gate"], post_stats=ps, pre_stats=qs)
    kw = dict(dpost_beta=g[1], dpre_beta=g[3]) if beta else {}
    elf.block_norm_bwd(nm, y, dx, dy=t["dy"], dh=t["dh"], f=t["f"], gate=t["gate"], df=df, dgate=dg, post_stats=ps,
                       pre_stats=qs, dpost_gamma=g[0], dpre_gamma=g[2], **kw)
    n = {k: np64(v) for k, v in t.items()}
    ref = bp.block_norm_fwd(n["x"], n["f"], n["gate"], "layer", "layer", n["gp"], n["bp"], n["gq"], n["bq"], act, gr, 0.5,
                            np.float64(np.float32(1e-5)), DT[dt])
    tp.check(y, ref["y"], "y")
    tp.check(h, ref["h"], "h")
    ref = bp.block_norm_bwd(n["dy"], n["dh"], np64(y), n["f"], n["gate"], "layer", "layer", n["gp"], n["bp"], n["gq"], n["bq"],
                            act, gr, 0.5, np64(ps), np64(qs), DT[dt])
    got = dict(dx=dx, df=df, dgate=dg, dpost_gamma=g[0], dpre_gamma=g[2])
    got.update(dict(dpost_beta=g[1], dpre_beta=g[3]) if beta else {})
    for k, v in got.items():
        tp.check(v, ref[k], k)
    assert all(gap_untouched(v) for v in (y, h, dx, df, dg))

"""Plain 64-bit forms of the residual block's operators (numpy), and the bounds that a 32-bit
computation with one rounding at the end keeps to.

Bounds.  u = 2^-24 is half a step of fp32, as in tests/tower_plain.py.
  * Packing is exact but for the rounding that defines it: codes and scale bytes have to be equal.
  * A sum over a row's C values is taken in fp32 in lanes' sums (at most 32 values behind each
    other), six exchanges and at most 16 wavefronts' sums: at most 64 additions behind each other,
    G = 64 u times the sum of the absolute values.
  * A sum over M rows adds at most M + 64 values behind each other.
  * exp2 of a rounded argument, a sum and a reciprocal give the sigmoid within (4 + 2 |v|) u of
    itself (the argument's error u |v| log2(e) enters as its relative error).
  * Block-scaled products of 4-bit numbers are exact; every addition of the K products is off by at
    most one step, 2 u.
"""
import numpy as np

from tests import tower_plain as tp
from tests.tower_plain import U, store_err

G = 64 * U
TINY = 2.0 ** -140


# ------------------------------------------------------------------ microscaled numbers
def numbers(exp_bits, frac_bits, count):
    """The first `count` magnitudes of a small float format, by code."""
    bias = 2 ** (exp_bits - 1) - 1
    out = []
    for code in range(count):
        ex, fr = code >> frac_bits, (code & (2**frac_bits - 1)) / 2**frac_bits
        out.append(fr * 2.0 ** (1 - bias) if ex == 0 else (1 + fr) * 2.0 ** (ex - bias))
    return np.array(out)


E4M3, E2M1 = numbers(4, 3, 127), numbers(2, 1, 8)


def nearest(q, table):
    """Codes of the nearest magnitudes, even codes at ties (q from 0 to the largest)."""
    hi = np.clip(np.searchsorted(table, q), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = q - table[lo], table[hi] - q
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def pack(x, fp4):
    """(codes [M, Kp] one per value with the sign bit, scale bytes [M, Kp / 32]) of float64 x."""
    table, pad = (E2M1, 128) if fp4 else (E4M3, 32)
    M, K = x.shape
    kp = -(-K // pad) * pad
    v = np.zeros((M, kp))
    v[:, :K] = x
    b = v.reshape(M, -1, 32)
    fin = np.isfinite(b)
    amax = np.where(fin, np.abs(b), 0.0).max(-1)
    e = np.full(amax.shape, -126)
    for t in range(-126, 128):  # the smallest exponent that holds the block
        e = np.where(amax > table[-1] * 2.0**t, t + 1, e)
    q = np.where(fin, np.abs(b), 0.0) / 2.0 ** e[..., None].astype(float)
    code = nearest(q, table)
    sign = np.signbit(b)
    byte = (e + 127).astype(np.int64)
    if fp4:
        bad = ~fin.all(-1)
        code = np.where(bad[..., None], 0, code + 8 * sign)
        byte = np.where(bad, 255, byte)
    else:
        code = np.where(fin, code + 128 * sign, 127)
    return code.reshape(M, kp), byte


def values(code, byte, K, fp4):
    """float64 [M, K] that codes and scale bytes stand for."""
    M = code.shape[0]
    table = E2M1 if fp4 else np.append(E4M3, np.nan)
    half = len(table)
    v = np.where(code >= half, -1.0, 1.0) * table[code % half]
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(float) - 127))
    return (v.reshape(M, -1, 32) * s[..., None]).reshape(M, -1)[:, :K]


def rounded(x, fp4):
    return values(*pack(x, fp4), x.shape[1], fp4)


def dense_fp4(x4, w4, bias, kind, res, dtype):
    K = x4.shape[1]
    b = bias if bias is not None else np.zeros(w4.shape[0])
    z = x4 @ w4.T + b
    ez = 2 * (-(-K // 128) * 128 + 2) * U * (np.abs(x4) @ np.abs(w4).T + np.abs(b))
    y = tp.act(z, kind)
    ey = tp.SLOPE * ez + tp.act_err(z, kind) + 2 * U * np.abs(y)
    if res is not None:
        y = y + res
        ey = ey + U * np.abs(y)
    return y, ey + store_err(y, dtype)


# ------------------------------------------------------------------ block norm
def stats(v, kind, eps):
    """mean, rstd [M, 1]."""
    mean = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    d = v - mean
    return mean, 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)


def norm(v, ev, kind, eps):
    """The normalised rows, their bound, and the statistics with theirs, of v known within ev."""
    n = v.shape[1]
    mean, rstd = stats(v, kind, eps)
    em = G * np.abs(v).mean(1, keepdims=True) + ev.mean(1, keepdims=True) if kind == "layer" else np.zeros_like(mean)
    d = v - mean
    ed = ev + em + U * np.abs(d)
    # the variance: sums of (d + ed)^2
    rel = G + 4 * U + (2 * (np.abs(d) * ed).sum(1, keepdims=True) + (ed * ed).sum(1, keepdims=True)) / n * rstd**2
    if kind == "layer":  # a mean that is off by em moves the sum of squares by n em^2 only
        ev2 = ev + U * np.abs(d)
        rel = G + 4 * U + (2 * (np.abs(d) * ev2).sum(1, keepdims=True) + (ed * ed).sum(1, keepdims=True)) / n * rstd**2
    er = rstd * (0.51 * rel + 4 * U)
    vh = d * rstd
    return vh, rstd * ed + np.abs(d) * er + 2 * U * np.abs(vh), mean, em, rstd, er


def gate_of(gate, act, M, rows):
    if gate is None:
        return 1.0, 0.0, None
    idx = np.arange(M) // rows
    if act == "sigmoid":
        g = 1 / (1 + np.exp(-gate))
        return g[idx], (g * (4 + 2 * np.abs(gate)) * U)[idx], g
    return gate[idx], 0.0, gate


def block_norm_fwd(x, f, gate, post, pre, gp, bp, gq, bq, gate_act, gate_rows, scale, eps, dtype):
    """{name: (value, bound)} for y, h and the statistics ([M, 2])."""
    like = x if x is not None else f
    M, C = like.shape
    one, zero = np.ones(C), np.zeros(C)
    gp, bp, gq, bq = (d if v is None else v for v, d in ((gp, one), (bp, zero), (gq, one), (bq, zero)))
    out = {}
    y = x if x is not None else np.zeros((M, C))
    ey = np.zeros((M, C))
    if f is not None:
        fh, efh = f, np.zeros((M, C))
        if post != "none":
            fh, efh, m, em, r, er = norm(f, np.zeros((M, C)), post, eps)
            out["post_stats"] = (np.concatenate([m, r], 1), np.concatenate([em, er], 1) + TINY)
        t = fh * gp + bp
        et = np.abs(gp) * efh + 2 * U * (np.abs(fh * gp) + np.abs(bp))
        g, eg, _ = gate_of(gate, gate_act, M, gate_rows)
        y = y + scale * g * t
        ey = np.abs(scale) * (np.abs(g) * et + np.abs(t) * eg) + 3 * U * np.abs(scale * g * t) + U * (np.abs(y) + np.abs(y - scale * g * t))
        out["y"] = (y, ey + store_err(y, dtype))
    yh, eyh, m, em, r, er = norm(y, ey, pre, eps)
    out["pre_stats"] = (np.concatenate([m, r], 1), np.concatenate([em, er], 1) + TINY)
    h = yh * gq + bq
    out["h"] = (h, np.abs(gq) * eyh + 2 * U * (np.abs(yh * gq) + np.abs(bq)) + store_err(h, dtype))
    return out


def pull(g, eg, vh, kind, rstd):
    """Gradient at a norm's input from g at its output, and its bound."""
    if kind == "none":
        return g, eg
    avg = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    evh = 2 * U * np.abs(vh)
    m2 = avg(g * vh)
    e2 = avg(eg * np.abs(vh) + np.abs(g) * evh) + (G + 8 * U) * avg(np.abs(g * vh))
    m1, e1 = 0.0, 0.0
    if kind == "layer":
        m1, e1 = avg(g), avg(eg) + (G + 8 * U) * avg(np.abs(g))
    d = rstd * (g - m1 - vh * m2)
    ed = rstd * (eg + e1 + np.abs(vh) * e2 + evh * np.abs(m2) + 8 * U * (np.abs(g) + np.abs(m1) + np.abs(vh * m2)))
    return d, ed


def block_norm_bwd(dy, dh, y, f, gate, post, pre, gp, bp, gq, bq, gate_act, gate_rows, scale, post_stats, pre_stats, dtype):
    """{name: (value, bound)} of every gradient; statistics [M, 2] as the kernels are given them."""
    like = dh if dh is not None else dy
    M, C = like.shape
    one, zero = np.ones(C), np.zeros(C)
    gp, bp, gq, bq = (d if v is None else v for v, d in ((gp, one), (bp, zero), (gq, one), (bq, zero)))
    rows = (M + 64) * U
    colsum = lambda a, ea: (a.sum(0), ea.sum(0) + rows * np.abs(a).sum(0) + TINY)  # noqa: E731
    out = {}
    D, eD = np.zeros((M, C)), np.zeros((M, C))
    if dh is not None:
        mean, rstd = pre_stats[:, :1], pre_stats[:, 1:]
        yh = (y - mean) * rstd
        out["dpre_gamma"] = colsum(dh * yh, 3 * U * np.abs(dh * yh))
        out["dpre_beta"] = colsum(dh, np.zeros_like(dh))
        a = dh * gq
        D, eD = pull(a, U * np.abs(a), yh, pre, rstd)
    if dy is not None:
        eD = eD + U * (np.abs(dy + D) + np.abs(D))
        D = D + dy
    out["dx"] = (D, eD + store_err(D, dtype))
    if f is None:
        return out
    mean, rstd = (post_stats[:, :1], post_stats[:, 1:]) if post != "none" else (0.0, 1.0)
    fh = (f - mean) * rstd
    efh = 2 * U * np.abs(fh)
    g, eg, graw = gate_of(gate, gate_act, M, gate_rows)
    sD, esD = scale * D, np.abs(scale) * eD + U * np.abs(scale * D)
    u = g * sD
    eu = np.abs(g) * esD + eg * np.abs(sD) + U * np.abs(u)
    out["dpost_gamma"] = colsum(u * fh, eu * np.abs(fh) + np.abs(u) * efh + U * np.abs(u * fh))
    out["dpost_beta"] = colsum(u, eu)
    b = u * gp
    out["df"] = pull(b, np.abs(gp) * eu + U * np.abs(b), fh, post, rstd)
    out["df"] = (out["df"][0], out["df"][1] + store_err(out["df"][0], dtype))
    if gate is not None:
        t = fh * gp + bp
        et = np.abs(gp) * efh + 2 * U * (np.abs(fh * gp) + np.abs(bp))
        p, ep = sD * t, esD * np.abs(t) + np.abs(sD) * et + U * np.abs(sD * t)
        R = -(-M // gate_rows)
        s, es, ab = (np.zeros((R, C)) for _ in range(3))
        for dst, src in ((s, p), (es, ep), (ab, np.abs(p))):
            np.add.at(dst, np.arange(M) // gate_rows, src)
        es = es + (min(gate_rows, M) + 64) * U * ab
        if gate_act == "sigmoid":
            d1 = graw * (1 - graw)
            es = np.abs(d1) * es + np.abs(s) * (graw * (12 + 4 * np.abs(gate)) * U)
            s = s * d1
        out["dgate"] = (s, es + store_err(s, dtype) + TINY)
    return out

"""Plain 64-bit forms of the dense-tower operators (numpy), their analytic gradients, and the
bounds that a 32-bit computation with one rounding at the end keeps to.

Bounds.  u = 2^-24 is half a step of fp32, h(t) half a step of the output type (finfo.eps / 2).
  * a sum of n products accumulated in fp32 in any order is off by at most (n + 2) u times the
    sum of the products' absolute values; sums that the group norm adds in trees (at most 512
    additions behind each other at the sizes tested) by 512 u;
  * an activation or its derivative passes an input error on times at most 1.13 (the largest
    slope of GELU; |act''| <= 1.2 for the derivatives) and adds at most 16 fp32 steps, 2^-20,
    of its own (exp2 of a rounded argument, a reciprocal and a polynomial of a few operations);
  * storing adds h(t) of the value, or half the smallest subnormal.
"""
import numpy as np
import torch

U = 2.0 ** -24
ACT_ERR = 2.0 ** -20
SLOPE, CURVE = 1.13, 1.2
GAMMA_GN = 512 * U


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def store_err(v, dtype):
    f = torch.finfo(dtype)
    return np.abs(v) * (f.eps / 2) * (1 + 2 * f.eps) + f.smallest_normal * f.eps / 2


def erf(x):
    return torch.erf(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def act(u, kind):
    if kind == "relu":
        return np.where(u > 0, u, 0.0)
    if kind == "gelu":
        return u * 0.5 * (1 + erf(u / np.sqrt(2)))
    if kind == "silu":
        return u / (1 + np.exp(-u))
    return u


def act_grad(u, kind):
    if kind == "relu":
        return (u > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * (1 + erf(u / np.sqrt(2))) + u * np.exp(-u * u / 2) / np.sqrt(2 * np.pi)
    if kind == "silu":
        s = 1 / (1 + np.exp(-u))
        return s * (1 + u * (1 - s))
    return np.ones_like(u)


def act_err(u, kind):
    """What the activation itself may add to an fp32 result at u."""
    return np.abs(u) * ACT_ERR if kind in ("gelu", "silu") else np.zeros_like(u)


def act_grad_err(u, kind):
    return (1 + np.abs(u)) * ACT_ERR if kind in ("gelu", "silu") else np.zeros_like(u)


def philox4x32_10(c, k):
    """Philox4x32-10 of the counter (4 uint64 arrays holding 32-bit words) under the key."""
    c = [np.asarray(v, np.uint64) for v in c]
    k0, k1 = int(k[0]), int(k[1])
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k0), p1 & low, (p0 >> sh) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def drop_factors(M, N, p, seed, offset):
    """[M, N] multipliers: 0 (dropped) or 65536 / (65536 - T)."""
    T = int(np.rint(p * 65536))
    if T == 65536:
        return np.zeros((M, N))
    g = np.arange((N + 7) // 8, dtype=np.uint64)
    rows = np.arange(M, dtype=np.uint64)
    ones = np.ones((M, g.size), np.uint64)
    offset &= 2**64 - 1
    w = philox4x32_10([ones * g[None, :], ones * rows[:, None], ones * np.uint64(offset & 0xFFFFFFFF),
                       ones * np.uint64(offset >> 32)], (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    bits = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], -1)
    keep = bits.reshape(M, -1)[:, :N] >= T
    return np.where(keep, 65536.0 / (65536 - T), 0.0)


def apply_drop(v, f):
    """v times the factors; a dropped value is 0 whatever it held."""
    if f is None:
        return v
    return np.where(f > 0, np.where(f > 0, v, 0.0) * f, 0.0)


def fmax(f):
    return 1.0 if f is None else float(max(1.0, np.max(f, initial=0.0)))


# ------------------------------------------------------------------ act_dropout
def act_dropout_fwd(x, kind, f, res, dtype):
    y = apply_drop(act(x, kind), f)
    err = fmax(f) * (act_err(x, kind) + 2 * U * np.abs(act(x, kind)))
    if res is not None:
        y = y + res
        err = err + U * np.abs(y)
    return y, err + store_err(y, dtype)


def act_dropout_bwd(dy, x, kind, f, dtype):
    g = act_grad(x, kind) if x is not None else np.ones_like(dy)
    ge = act_grad_err(x, kind) if x is not None else 0.0
    dx = apply_drop(dy * g, f)
    err = fmax(f) * np.abs(dy) * (ge + 3 * U * np.abs(g))
    return dx, err + store_err(dx, dtype)


# ------------------------------------------------------------------ dense
def dense_fwd(x, w, bias, kind, f, res, dtype):
    K = x.shape[1]
    b = bias if bias is not None else np.zeros(w.shape[0])
    z = x @ w.T + b
    ez = (K + 2) * U * (np.abs(x) @ np.abs(w).T + np.abs(b))
    y = apply_drop(act(z, kind), f)
    ey = fmax(f) * (SLOPE * ez + act_err(z, kind) + 2 * U * np.abs(act(z, kind)))
    if res is not None:
        y = y + res
        ey = ey + U * np.abs(y)
    return y, ey + store_err(y, dtype), z, ez + store_err(z, dtype)


def dense_bwd(x, w, dz, dres, pre, kind, f, dtype):
    M, N = dz.shape
    dx = dz @ w
    ex = (N + 2) * U * (np.abs(dz) @ np.abs(w))
    if dres is not None:
        dx = dx + dres
        ex = ex + U * (np.abs(dx) + np.abs(dres))
    g = act_grad(pre, kind) if pre is not None else np.ones_like(dx)
    ge = act_grad_err(pre, kind) if pre is not None else 0.0
    dzb = apply_drop(dx * g, f)
    eb = fmax(f) * (SLOPE * ex + np.abs(dx) * (ge + 3 * U))
    dw, db = dz.T @ x, dz.sum(0)
    ew, ebias = (M + 2) * U * (np.abs(dz).T @ np.abs(x)), (M + 2) * U * np.abs(dz).sum(0)
    tiny = 2.0 ** -140
    return dict(dx=(dx, ex + store_err(dx, dtype)), dzb=(dzb, eb + store_err(dzb, dtype)), dw=(dw, ew + tiny),
                db=(db, ebias + tiny))


# ------------------------------------------------------------------ group norm
def _valid(B, S, lengths):
    n = np.full(B, S) if lengths is None else np.clip(lengths, 0, S)
    return n, (np.arange(S)[None, :] < n[:, None])[:, :, None, None]


def gn_stats(x, S, G, lengths, eps):
    """mean, rstd [B, G] and their bounds; x [B*S, C]."""
    C = x.shape[1]
    B = x.shape[0] // S
    n, ok = _valid(B, S, lengths)
    v = np.where(ok, x.reshape(B, S, G, C // G), 0.0)
    cnt = np.maximum(n, 1)[:, None] * (C // G)
    mean = v.sum((1, 3)) / cnt
    d = np.where(ok, v - mean[:, None, :, None], 0.0)
    var = (d * d).sum((1, 3)) / cnt
    rstd = 1 / np.sqrt(var + eps)
    em = GAMMA_GN * np.abs(v).sum((1, 3)) / cnt
    er = rstd * (GAMMA_GN + 8 * U + rstd**2 * em * (em + 2 * U * np.abs(v).max((1, 3), initial=0)))
    return mean, rstd, em, er


def gn_fwd(x, S, G, lengths, gamma, beta, eps, kind, dtype):
    C = x.shape[1]
    B = x.shape[0] // S
    n, ok = _valid(B, S, lengths)
    mean, rstd, em, er = gn_stats(x, S, G, lengths, eps)
    ex4 = lambda a: a[:, None, :, None]  # noqa: E731
    v = np.where(ok, x.reshape(B, S, G, C // G), 0.0)
    gm = (np.ones(C) if gamma is None else gamma).reshape(G, -1)
    bt = (np.zeros(C) if beta is None else beta).reshape(G, -1)
    xh = (v - ex4(mean)) * ex4(rstd)
    exh = ex4(rstd) * (ex4(em) + U * (np.abs(v) + np.abs(ex4(mean)))) * 2 + np.abs(v - ex4(mean)) * ex4(er)
    u = gm * xh + bt
    eu = np.abs(gm) * exh + 3 * U * (np.abs(gm * xh) + np.abs(bt))
    y = np.where(ok, act(u, kind), 0.0)
    ey = SLOPE * eu + act_err(u, kind)
    y, ey = y.reshape(B * S, C), np.where(ok, ey, 0.0).reshape(B * S, C)
    return y, ey + store_err(y, dtype), (mean, em + 1e-37), (rstd, er)


def gn_bwd(dy, x, S, G, lengths, gamma, beta, mean, rstd, kind, dtype):
    C = x.shape[1]
    B = x.shape[0] // S
    n, ok = _valid(B, S, lengths)
    ex4 = lambda a: a[:, None, :, None]  # noqa: E731
    shape = (B, S, G, C // G)
    v = np.where(ok, x.reshape(shape), ex4(mean))
    d = np.where(ok, dy.reshape(shape), 0.0)
    gm = (np.ones(C) if gamma is None else gamma).reshape(G, -1)
    bt = (np.zeros(C) if beta is None else beta).reshape(G, -1)
    xh = (v - ex4(mean)) * ex4(rstd)
    exh = 2 * U * (ex4(rstd) * (np.abs(v) + np.abs(ex4(mean))) + np.abs(xh))
    u = gm * xh + bt
    eu = np.abs(gm) * exh + 3 * U * (np.abs(gm * xh) + np.abs(bt))
    du = d * act_grad(u, kind)
    edu = np.abs(d) * (CURVE * eu + act_grad_err(u, kind)) + U * np.abs(du)
    if kind == "relu":  # either side of the border is right within the error of u
        edu = np.where(np.abs(u) <= eu, np.abs(d), U * np.abs(du))
    if kind == "none":
        edu = U * np.abs(du)
    dh, edh = du * gm, np.abs(gm) * edu + U * np.abs(du * gm)
    cnt = ex4(np.maximum(n, 1)[:, None] * (C // G))
    avg = lambda a: a.sum((1, 3), keepdims=True) / cnt  # noqa: E731
    m1, m2 = avg(dh), avg(dh * xh)
    e1 = avg(edh) + GAMMA_GN * avg(np.abs(dh))
    e2 = avg(edh * np.abs(xh) + np.abs(dh) * exh) + GAMMA_GN * avg(np.abs(dh * xh))
    r = ex4(rstd)
    dx = r * (dh - m1 - xh * m2)
    edx = r * (edh + e1 + np.abs(xh) * e2 + exh * np.abs(m2) + 6 * U * (np.abs(dh) + np.abs(m1) + np.abs(xh * m2)))
    dx, edx = np.where(ok, dx, 0.0).reshape(B * S, C), np.where(ok, edx, 0.0).reshape(B * S, C)
    s = lambda a: a.sum((0, 1)).reshape(C)  # noqa: E731
    big = 1024 * U
    dg, eg = s(du * xh), s(edu * np.abs(xh) + np.abs(du) * exh) + big * s(np.abs(du * xh))
    db, eb = s(du), s(edu) + big * s(np.abs(du))
    return dict(dx=(dx, edx + store_err(dx, dtype)), dgamma=(dg, eg + 1e-37), dbeta=(db, eb + 1e-37))


# ------------------------------------------------------------------ comparison
def check(got: torch.Tensor, want, what):
    ref, tol = want
    g = got.detach().double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(g).all(), f"{what}: {np.sum(~np.isfinite(g))} values not finite"
    bad = np.abs(g - ref) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(g - ref) / np.maximum(tol, 1e-300)), ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound; worst at {i}: got {g[i]!r}, "
                             f"want {ref[i]!r}, bound {np.broadcast_to(tol, ref.shape)[i]!r}")

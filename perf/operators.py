"""Cases and plain forms of the dense-tower operators: what they compute, on which sizes, and
what one pass has to move and multiply.

The operators are the parts of a deeper tower on top of the pooled embeddings:
  dense       y = residual + dropout(act(x w^T + bias)), and its gradients;
  act_dropout y = residual + dropout(act(x)), and its gradient;
  group_norm  y = act(gamma (x - mean) rstd + beta) over groups of channels, channels last,
              and its gradients.
The dropout mask is a function of (seed, offset, row, column) and is never stored: Philox4x32-10
(Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) on the counter
(column / 8, row, offset low, offset high) under the key (seed low, seed high) gives eight
16-bit numbers, one per column of the group, low half of a word first; a value is kept where
its number is >= T = round(65536 p), and then scaled by 65536 / (65536 - T).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
ROWS, WIDTH = 65536, 1024  # the largest batch and the widest layer of the model's top MLP
GN_ELEMENTS = 16384 * 26 * 128


def listed():
    return [
        # one candidate scored by the 1024-wide residual layer of the top MLP: latency
        dict(name="dense_fwd_one_row", op="dense_fwd", M=1, K=1024, N=1024, dtype="bf16",
             act="gelu", p=0.0, residual=True, pre=False, extra=0),
        # a ragged handful of candidates through the top MLP's first layer (interaction output
        # kept 512 wide)
        dict(name="dense_fwd_77_rows", op="dense_fwd", M=77, K=512, N=1024, dtype="f16",
             act="silu", p=0.0, residual=False, pre=False, extra=0),
        # the training forward of the widest layer at the full batch: residual, dropout, and
        # the pre-activation kept for the backward
        dict(name="dense_fwd_train", op="dense_fwd", M=ROWS, K=1024, N=1024, dtype="bf16",
             act="gelu", p=0.1, residual=True, pre=True, extra=0),
        # the last, ragged batch of an epoch through the unpadded interaction output: 479
        # columns in rows of 512
        dict(name="dense_fwd_odd", op="dense_fwd", M=4099, K=479, N=1001, dtype="bf16",
             act="relu", p=0.25, residual=True, pre=True, extra=33),
        # its backward at the full batch: weight, bias and data gradients, the skip
        # connection's gradient added and the layer below's activation and dropout undone
        dict(name="dense_bwd_train", op="dense_bwd", M=ROWS, K=1024, N=1024, dtype="bf16",
             act="gelu", p=0.1, residual=True, extra=0),
        # the backward of a bottom layer on a ragged batch
        dict(name="dense_bwd_ragged", op="dense_bwd", M=4099, K=512, N=256, dtype="f16",
             act="silu", p=0.5, residual=False, extra=8),
        # dropout alone on a small batch's pooled vectors: latency
        dict(name="act_dropout_fwd_small", op="act_dropout_fwd", M=64, N=128, dtype="bf16",
             act="none", p=0.2, residual=False, extra=0),
        # activation, dropout and residual over a whole layer's output
        dict(name="act_dropout_fwd_train", op="act_dropout_fwd", M=ROWS, N=1024, dtype="bf16",
             act="gelu", p=0.1, residual=True, extra=0),
        # the gradient over the unpadded 479-wide interaction output, in rows of 512
        dict(name="act_dropout_bwd_odd", op="act_dropout_bwd", M=16411, N=479, dtype="f32",
             act="silu", p=0.3, residual=False, extra=33),
        # a few samples' pooled vectors (26 tables of 128) normalised before the interaction
        dict(name="group_norm_fwd_small", op="group_norm_fwd", M=64, S=26, C=128, G=8, dtype="bf16",
             act="none", ragged=False, extra=0),
        # the same in training, forward and backward
        dict(name="group_norm_train", op="group_norm_train", M=16384, S=26, C=128, G=8, dtype="bf16",
             act="silu", ragged=False, extra=0),
        # long padded histories of a few users, each with a length of its own
        dict(name="group_norm_train_long", op="group_norm_train", M=6, S=5001, C=256, G=32, dtype="f16",
             act="silu", ragged=True, extra=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dense_fwd", "dense_bwd", "act_dropout_fwd", "act_dropout_bwd", "group_norm_fwd",
                     "group_norm_train"])
    c = dict(op=op, act=rng.choice(["none", "relu", "gelu", "silu"]), extra=rng.choice([0, 0, 8, 24]))
    if op.startswith("group_norm"):
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["G"] = rng.choice([1, 2, 4, 8, 16, 32])
        c["C"] = c["G"] * _log(rng, 1, 64)
        c["S"] = _log(rng, 1, 8192)
        c["C"] = max(c["C"], c["G"] * -(-16 // c["S"]))  # 16 values at least behind each mean
        if op == "group_norm_train" and c["act"] == "relu":
            c["act"] = "silu"  # ReLU's gradient jumps where two right roundings may part
        c["M"] = _log(rng, 1, max(1, min(ROWS, GN_ELEMENTS // (2 * c["S"] * c["C"]))))
        c["ragged"] = rng.random() < 0.5
        return c
    c["p"] = rng.choice([0.0, 0.1, 0.25, 0.5])
    c["residual"] = rng.random() < 0.5
    c["M"] = _log(rng, 1, ROWS)
    c["N"] = _log(rng, 1, WIDTH)
    if op.startswith("act_dropout"):
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        return c
    c["dtype"] = rng.choice(["bf16", "f16"])
    c["K"] = _log(rng, 1, WIDTH)
    if rng.random() < 0.75:  # most layers are padded to whole vectors
        c["N"], c["K"] = (c["N"] + 7) // 8 * 8, (c["K"] + 7) // 8 * 8
    if op == "dense_fwd":
        c["pre"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------------------
# Inputs and the buffers a training or serving program keeps.
# ---------------------------------------------------------------------------------------
def _rows(g, m, n, extra, dtype, scale=1.0, shift=0.0):
    """[m, n] normal values as the first n columns of rows n + extra wide."""
    t = torch.randn((m, n + extra), generator=g, device=g.device)
    return t.mul_(scale).add_(shift).to(DTYPES[dtype])[:, :n]


def _out(m, n, extra, dtype, device):
    return torch.empty((m, n + extra), dtype=DTYPES[dtype], device=device)[:, :n]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    c, op, dt, ex = case, case["op"], case["dtype"], case["extra"]
    s = dict(case=dict(case), seed=1_000_003 * int(seed) + 12345, offset=int(seed) % 1000)
    if op.startswith("group_norm"):
        M, S, C, G = c["M"], c["S"], c["C"], c["G"]
        s["x"] = _rows(g, M * S, C, ex, dt, 1.0, 0.5)
        s["gamma"] = 1.0 + 0.1 * torch.randn(C, generator=g, device=dev)
        s["beta"] = 0.1 * torch.randn(C, generator=g, device=dev)
        # lengths of the padded histories, none and full among them
        s["lengths"] = torch.randint(0, S + 1, (M,), generator=g, device=dev, dtype=torch.int32) if c["ragged"] else None
        s["y"] = _out(M * S, C, ex, dt, dev)
        s["mean"] = torch.empty((M, G), device=dev)
        s["rstd"] = torch.empty((M, G), device=dev)
        if op == "group_norm_train":
            s["dy"] = _rows(g, M * S, C, ex, dt)
            s["dx"] = _out(M * S, C, ex, dt, dev)
            s["dgamma"] = torch.empty(C, device=dev)
            s["dbeta"] = torch.empty(C, device=dev)
            s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
        else:
            s["workspace"] = torch.empty(8 << 20, dtype=torch.uint8, device=dev)
        return s
    M, N = c["M"], c["N"]
    if op == "act_dropout_fwd":
        s["x"] = _rows(g, M, N, ex, dt)
        s["residual"] = _rows(g, M, N, ex, dt) if c["residual"] else None
        s["y"] = _out(M, N, ex, dt, dev)
        return s
    if op == "act_dropout_bwd":
        s["dy"] = _rows(g, M, N, ex, dt)
        s["pre"] = _rows(g, M, N, ex, dt)
        s["dx"] = _out(M, N, ex, dt, dev)
        return s
    K = c["K"]
    s["x"] = _rows(g, M, K, ex, dt)
    s["w"] = _rows(g, N, K, 0, dt, 1.0 / math.sqrt(K))
    if op == "dense_fwd":
        s["bias"] = 0.1 * torch.randn(N, generator=g, device=dev)
        s["residual"] = _rows(g, M, N, ex, dt) if c["residual"] else None
        s["pre"] = _out(M, N, ex, dt, dev) if c["pre"] else None
        s["y"] = _out(M, N, ex, dt, dev)
        s["workspace"] = torch.empty(160 << 20, dtype=torch.uint8, device=dev)
        return s
    s["dz"] = _rows(g, M, N, ex, dt)
    s["dres"] = _rows(g, M, K, ex, dt) if c["residual"] else None
    s["pre"] = _rows(g, M, K, ex, dt)
    s["dx"] = _out(M, K, ex, dt, dev)
    s["dzb"] = _out(M, K, ex, dt, dev)
    s["dw"] = torch.empty((N, K), device=dev)
    s["db"] = torch.empty(N, device=dev)
    s["workspace"] = torch.empty(512 << 20, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------------------
_LOW = 0xFFFFFFFF


def _keep(m, n, p, seed, offset, device):
    """([m, n] kept?, scale) of the dropout mask."""
    t = round(65536 * p)
    col = torch.arange((n + 7) // 8, dtype=torch.int64, device=device)
    row = torch.arange(m, dtype=torch.int64, device=device)
    c0 = col[None, :].expand(m, -1)
    c1 = row[:, None].expand(-1, col.numel())
    c2 = torch.full_like(c0, offset & _LOW)
    c3 = torch.full_like(c0, (offset >> 32) & _LOW)
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):  # the generator's rounds; int64 products wrap, which keeps their 64 bits
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    words = torch.stack([c0, c1, c2, c3], dim=-1)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=-1).reshape(m, -1)[:, :n]
    return bits >= t, (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _act(u, act):
    if act == "relu":
        return torch.where(u > 0, u, torch.zeros_like(u))
    if act == "gelu":
        return 0.5 * u * (1.0 + torch.erf(u * (1.0 / math.sqrt(2.0))))
    if act == "silu":
        return u / (1.0 + torch.exp(-u))
    return u


def _act_grad(u, act):
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(u * (1.0 / math.sqrt(2.0)))) + u * torch.exp(-0.5 * u * u) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-u))
        return s * (1.0 + u * (1.0 - s))
    return torch.ones_like(u)


def _drop(a, s):
    c = s["case"]
    if c["p"] == 0.0:
        return a
    keep, scale = _keep(a.shape[0], a.shape[1], c["p"], s["seed"], s["offset"], a.device)
    return torch.where(keep, a * scale, torch.zeros_like(a))


def _plain_dense_fwd(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    z = s["x"].float() @ s["w"].float().t() + s["bias"]
    y = _drop(_act(z, c["act"]), s)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    out = {"y": y.to(dt)}
    if c["pre"]:
        out["pre"] = z.to(dt)
    return out


def _plain_dense_bwd(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    dz = s["dz"].float()
    dx = dz @ s["w"].float()
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    dzb = _drop(dx * _act_grad(s["pre"].float(), c["act"]), s)
    return {"dx": dx.to(dt), "dzb": dzb.to(dt), "dw": dz.t() @ s["x"].float(), "db": dz.sum(0)}


def _plain_group_norm(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    M, S, C, G = c["M"], c["S"], c["C"], c["G"]
    shape = (M, S, G, C // G)
    x = s["x"].float().reshape(shape)
    gamma, beta = s["gamma"].view(G, -1), s["beta"].view(G, -1)
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((M,), S, device=x.device)
    valid = (torch.arange(S, device=x.device)[None, :] < lengths[:, None]).view(M, S, 1, 1)
    count = (lengths.clamp(min=1) * (C // G)).float().view(M, 1, 1, 1)
    zero = torch.zeros((), device=x.device)
    x = torch.where(valid, x, zero)
    mean = x.sum((1, 3), keepdim=True) / count
    d = torch.where(valid, x - mean, zero)
    rstd = 1.0 / torch.sqrt((d * d).sum((1, 3), keepdim=True) / count + EPS)
    xh = d * rstd
    u = xh * gamma + beta
    y = torch.where(valid, _act(u, c["act"]), zero)
    out = {"y": y.reshape(M * S, C).to(dt), "mean": mean.view(M, G), "rstd": rstd.view(M, G)}
    if c["op"] == "group_norm_train":
        du = torch.where(valid, s["dy"].float().reshape(shape) * _act_grad(u, c["act"]), zero)
        dh = du * gamma
        m1 = dh.sum((1, 3), keepdim=True) / count
        m2 = (dh * xh).sum((1, 3), keepdim=True) / count
        dx = torch.where(valid, rstd * (dh - m1 - xh * m2), zero)
        out["dx"] = dx.reshape(M * S, C).to(dt)
        out["dgamma"] = (du * xh).sum((0, 1)).reshape(C)
        out["dbeta"] = du.sum((0, 1)).reshape(C)
    return out


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "dense_fwd":
        return _plain_dense_fwd(s)
    if op == "dense_bwd":
        return _plain_dense_bwd(s)
    if op.startswith("group_norm"):
        return _plain_group_norm(s)
    dt = DTYPES[c["dtype"]]
    if op == "act_dropout_fwd":
        y = _drop(_act(s["x"].float(), c["act"]), s)
        if s["residual"] is not None:
            y = s["residual"].float() + y
        return {"y": y.to(dt)}
    return {"dx": _drop(s["dy"].float() * _act_grad(s["pre"].float(), c["act"]), s).to(dt)}


# ---------------------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------------------
def _own(s):
    import embedding_lookup_feature_amd as elf

    c, op = s["case"], s["case"]["op"]
    if op.startswith("group_norm"):
        elf.group_norm_fwd(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], positions=c["S"],
                           groups=c["G"], eps=EPS, act=c["act"], lengths=s["lengths"], workspace=s["workspace"])
        out = {k: s[k] for k in ("y", "mean", "rstd")}
        if op == "group_norm_train":
            elf.group_norm_bwd(s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], s["dx"],
                               s["dgamma"], s["dbeta"], positions=c["S"], groups=c["G"], act=c["act"],
                               lengths=s["lengths"], workspace=s["workspace"])
            out.update({k: s[k] for k in ("dx", "dgamma", "dbeta")})
        return out
    drop = elf.Dropout(c["p"], s["seed"], s["offset"]) if c["p"] > 0.0 else None
    if op == "dense_fwd":
        elf.dense_fwd(s["x"], s["w"], s["bias"], s["y"], act=c["act"], dropout=drop, residual=s["residual"],
                      pre=s["pre"], workspace=s["workspace"])
        return {"y": s["y"], "pre": s["pre"]} if c["pre"] else {"y": s["y"]}
    if op == "dense_bwd":
        elf.dense_bwd(s["x"], s["w"], s["dz"], s["dw"], s["db"], dx=s["dx"], dres=s["dres"], dzb=s["dzb"],
                      pre=s["pre"], act=c["act"], dropout=drop, workspace=s["workspace"])
        return {k: s[k] for k in ("dx", "dzb", "dw", "db")}
    if op == "act_dropout_fwd":
        elf.act_dropout_fwd(s["x"], s["y"], act=c["act"], dropout=drop, residual=s["residual"])
        return {"y": s["y"]}
    elf.act_dropout_bwd(s["dy"], s["pre"], s["dx"], act=c["act"], dropout=drop)
    return {"dx": s["dx"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------------------
def work(case):
    c, op, e = case, case["op"], SIZE[case["dtype"]]
    if op.startswith("group_norm"):
        n = c["M"] * c["S"] * c["C"]
        if c["ragged"]:  # half the positions are padding: their inputs are not needed, their outputs are zeros
            read, flops = n // 2, 10 * (n // 2)
        else:
            read, flops = n, 10 * n
        small = 8 * c["C"] + 8 * c["M"] * c["G"]
        if op == "group_norm_fwd":
            return {"bytes": e * (read + n) + small, "flops": flops}
        return {"bytes": e * (2 * read + 2 * n) + 2 * small, "flops": 3 * flops}
    mn = c["M"] * c["N"]
    if op == "act_dropout_fwd":
        return {"bytes": e * mn * (3 if c["residual"] else 2), "flops": 10 * mn}
    if op == "act_dropout_bwd":
        return {"bytes": e * mn * 3, "flops": 10 * mn}
    mk, nk = c["M"] * c["K"], c["N"] * c["K"]
    if op == "dense_fwd":
        b = e * (mk + nk + mn * (1 + int(c["residual"]) + int(c["pre"]))) + 4 * c["N"]
        return {"bytes": b, "flops": 2 * mk * c["N"]}
    b = e * (mk * (4 + int(c["residual"])) + nk + mn) + 4 * (nk + c["N"])
    return {"bytes": b, "flops": 4 * mk * c["N"]}


# ---------------------------------------------------------------------------------------
# The operators' definition in 64 bits, apart from the forms above.
# ---------------------------------------------------------------------------------------
def _exact_mask(m, n, p, seed, offset):
    """[m, n] factors (0 or the scale) of the dropout mask, by numpy's unsigned integers."""
    t = int(math.floor(65536 * p + 0.5))
    if t >= 65536:
        return np.zeros((m, n))
    groups = -(-n // 8)
    ctr = np.zeros((4, m, groups), dtype=np.uint64)
    ctr[0] = np.arange(groups, dtype=np.uint64)
    ctr[1] = np.arange(m, dtype=np.uint64)[:, None]
    ctr[2], ctr[3] = offset % 2**32, offset // 2**32 % 2**32
    low, sh = np.uint64(2**32 - 1), np.uint64(32)
    for r in range(10):
        ka = np.uint64((seed % 2**32 + r * 0x9E3779B9) % 2**32)
        kb = np.uint64((seed // 2**32 % 2**32 + r * 0xBB67AE85) % 2**32)
        pa, pb = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = np.stack([(pb >> sh) ^ ctr[1] ^ ka, pb & low, (pa >> sh) ^ ctr[3] ^ kb, pa & low])
    halves = np.moveaxis(ctr, 0, -1).astype(np.uint32)[..., None] >> np.array([0, 16], dtype=np.uint32)
    bits = (halves & np.uint32(0xFFFF)).reshape(m, groups * 8)[:, :n]
    return np.where(bits >= t, 65536.0 / (65536 - t), 0.0)


def _exact_act(u, act, grad=False):
    if act == "none":
        return np.ones_like(u) if grad else u
    if act == "relu":
        return np.heaviside(u, 0.0) if grad else np.maximum(u, 0.0)
    t = torch.from_numpy(np.ascontiguousarray(u))
    if act == "gelu":  # u Phi(u); Phi(u) + u phi(u)
        phi = torch.special.ndtr(t).numpy()
        return phi + u * np.exp(-u * u / 2) / np.sqrt(2 * np.pi) if grad else u * phi
    sig = torch.sigmoid(t).numpy()
    return sig + u * sig * (1 - sig) if grad else u * sig


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    h = {k: v.detach().cpu().double().numpy() if isinstance(v, torch.Tensor) and v.is_floating_point() and k not in
         ("y", "dx", "dzb", "dw", "db", "dgamma", "dbeta", "mean", "rstd") and not (k == "pre" and op == "dense_fwd")
         else v for k, v in s.items()}
    f64 = lambda v: torch.from_numpy(np.ascontiguousarray(v))  # noqa: E731
    if op.startswith("group_norm"):
        M, S, C, G = c["M"], c["S"], c["C"], c["G"]
        train = op == "group_norm_train"
        y = np.zeros((M, S, C))
        mean, rstd = np.zeros((M, G)), np.full((M, G), EPS ** -0.5)
        dx, dgamma, dbeta = (np.zeros((M, S, C)), np.zeros(C), np.zeros(C)) if train else (None, None, None)
        gam, bet = h["gamma"].reshape(G, -1), h["beta"].reshape(G, -1)
        lengths = s["lengths"].cpu().numpy() if s["lengths"] is not None else np.full(M, S)
        step = max(1, (1 << 21) // max(1, S * C)) if not c["ragged"] else 1
        if M // step > 20000:
            return None
        X, D = h["x"].reshape(M, S, C), h["dy"].reshape(M, S, C) if train else None
        for b in range(0, M, step):
            e = min(M, b + step)
            L = int(lengths[b])
            if L == 0:
                continue
            v = X[b:e, :L].reshape(e - b, L, G, C // G)
            mu = v.mean(axis=(1, 3), keepdims=True)
            r = 1 / np.sqrt(v.var(axis=(1, 3), keepdims=True) + EPS)
            xh = (v - mu) * r
            u = gam * xh + bet
            y[b:e, :L] = _exact_act(u, c["act"]).reshape(e - b, L, C)
            mean[b:e], rstd[b:e] = mu.reshape(e - b, G), r.reshape(e - b, G)
            if train:
                du = D[b:e, :L].reshape(v.shape) * _exact_act(u, c["act"], True)
                dgamma += (du * xh).sum(axis=(0, 1)).reshape(C)
                dbeta += du.sum(axis=(0, 1)).reshape(C)
                q = du * gam
                q = q - q.mean(axis=(1, 3), keepdims=True) - xh * (q * xh).mean(axis=(1, 3), keepdims=True)
                dx[b:e, :L] = (r * q).reshape(e - b, L, C)
        out = {"y": f64(y.reshape(M * S, C)), "mean": f64(mean), "rstd": f64(rstd)}
        if train:
            out.update(dx=f64(dx.reshape(M * S, C)), dgamma=f64(dgamma), dbeta=f64(dbeta))
        return out
    M, N = c["M"], c["N"]
    width = c["K"] if op == "dense_bwd" else N
    mask = _exact_mask(M, width, c["p"], s["seed"], s["offset"]) if c["p"] > 0 else 1.0
    pick = lambda v: np.where(mask > 0, v * mask, 0.0)  # noqa: E731
    if op == "act_dropout_fwd":
        y = pick(_exact_act(h["x"], c["act"]))
        return {"y": f64(y if h["residual"] is None else y + h["residual"])}
    if op == "act_dropout_bwd":
        return {"dx": f64(pick(h["dy"] * _exact_act(h["pre"], c["act"], True)))}
    wide = lambda k: s[k].double()  # noqa: E731  (the products in 64 bits where the inputs are)
    if op == "dense_fwd":
        z = (torch.mm(wide("x"), wide("w").t().contiguous()) + wide("bias")).cpu().numpy()
        y = pick(_exact_act(z, c["act"]))
        y = f64(y if h["residual"] is None else y + h["residual"])
        return {"y": y, "pre": f64(z)} if c["pre"] else {"y": y}
    dx = torch.mm(wide("dz"), wide("w")).cpu().numpy()
    if h["dres"] is not None:
        dx = dx + h["dres"]
    dzb = pick(dx * _exact_act(h["pre"], c["act"], True))
    dw = torch.mm(wide("dz").t().contiguous(), wide("x")).cpu()
    return {"dx": f64(dx), "dzb": f64(dzb), "dw": dw, "db": wide("dz").sum(0).cpu()}

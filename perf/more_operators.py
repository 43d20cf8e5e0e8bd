"""Cases and plain forms of the operators of a normalised residual block: what they compute, on
which sizes, and what one pass has to move and multiply.

  block_norm  t = post_gamma norm_post(f) + post_beta,  y = x + scale act(gate) t,
              h = pre_gamma norm_pre(y) + pre_beta, and all their gradients: the norms behind one
              block and before the next, with the block's gate and residual scale;
  ckpt        activations kept in 8 bits between the forward and the backward pass: stored,
              activation and dropout computed again from them, the activation's gradient, and the
              dense layer's backward that reads its input and its pre-activation from them;
  fp4         weights and activations in microscaled 4 bits, and the dense layer on them.

8 and 4 bits are the microscaled formats of the Open Compute Project: 32 consecutive columns of a
row share a power of two 2^e, e >= -126, the smallest for which the largest magnitude of the block
is at most 448 2^e (8 bits, e4m3) or 6 2^e (4 bits, e2m1); each value divided by it is rounded to
the nearest number of the format, ties to even.

The dropout mask is the tower's: Philox4x32-10 on (column / 8, row, offset low, offset high) under
(seed low, seed high), eight 16-bit numbers for eight columns, kept where the number is
>= T = round(65536 p) and scaled by 65536 / (65536 - T).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
BLOCK = 32
ROWS, WIDTH = 65536, 1024  # the largest batch and the widest layer of the model's top MLP


def listed():
    return [
        # one candidate scored by a residual block of the 1024-wide tower: latency
        dict(name="norm_fwd_one_row", op="norm_fwd", M=1, C=1024, dtype="bf16", post="rms", pre="rms", gate="none",
             gate_rows=1, scale=0.5, beta=False, stats=False, extra=0),
        # one residual block of the 1024-wide tower at the full training batch, its gate computed
        # by a layer of its own
        dict(name="norm_fwd_full_batch", op="norm_fwd", M=ROWS, C=WIDTH, dtype="bf16", post="rms", pre="rms",
             gate="sigmoid", gate_rows=1, scale=0.5, beta=False, stats=True, extra=0),
        # its backward
        dict(name="norm_bwd_full_batch", op="norm_bwd", M=ROWS, C=WIDTH, dtype="bf16", post="rms", pre="rms",
             gate="sigmoid", gate_rows=1, scale=0.5, beta=False, extra=0),
        # the pooled vectors of an odd batch, 26 tables of 128, normalised and gated sample by
        # sample: backward, the gate shared by a sample's 26 rows
        dict(name="norm_bwd_pooled", op="norm_bwd", M=16387 * 26, C=128, dtype="f16", post="layer", pre="layer",
             gate="plain", gate_rows=26, scale=1.0, beta=True, extra=0),
        # the interaction output (479 columns) of a ragged handful of samples: latency, odd sizes
        dict(name="ckpt_77_rows", op="ckpt", M=77, C=479, dtype="f16", act="none", p=0.0, extra=1),
        # the widest layer's pre-activation at the full training batch
        dict(name="ckpt_full_batch", op="ckpt", M=ROWS, C=WIDTH, dtype="bf16", act="gelu", p=0.1, extra=0),
        # backward of the widest layer at the full training batch, skip connection included
        dict(name="dense_bwd_ckpt_full_batch", op="dense_bwd_ckpt", M=ROWS, K=WIDTH, N=WIDTH, dtype="bf16", act="gelu",
             p=0.1, residual=True, extra=0),
        # backward of the layer behind the interaction for an odd batch, rows padded
        dict(name="dense_bwd_ckpt_ragged", op="dense_bwd_ckpt", M=4099, K=479, N=256, dtype="f16", act="silu", p=0.2,
             residual=False, extra=1),
        # a large table of weights packed for serving and read back
        dict(name="fp4_pack_large", op="fp4_pack", M=32768, K=WIDTH, dtype="bf16", extra=0),
        # one candidate through the tower's 1024-wide residual layer: latency
        dict(name="dense_fp4_one_row", op="dense_fp4", M=1, K=WIDTH, N=WIDTH, dtype="bf16", act="gelu", residual=True,
             refresh=False, extra=0),
        # an odd batch through the layer behind the interaction, odd widths, its weights updated by
        # the last training step and packed again (evaluation during training)
        dict(name="dense_fp4_ragged", op="dense_fp4", M=4099, K=479, N=1001, dtype="f16", act="relu", residual=False,
             refresh=True, extra=1),
        # the largest offline batch through the widest layer
        dict(name="dense_fp4_full_batch", op="dense_fp4", M=ROWS, K=WIDTH, N=WIDTH, dtype="bf16", act="gelu",
             residual=True, refresh=False, extra=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Rows from one to the full batch, widths from one column (norms: the narrowest embedding's 16)
    to several times the tower's, every type, norm, gate and activation; whole vectors as often as
    odd widths."""
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_bwd", "ckpt", "dense_bwd_ckpt", "fp4_pack", "dense_fp4"])
    whole = rng.random() < 0.5
    width = lambda hi, lo=1: (lambda v: (v + 7) // 8 * 8 if whole else v)(_log(rng, lo, hi))  # noqa: E731
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), extra=rng.choice([0, 0, 0, 1, 8]))
    if op in ("norm_fwd", "norm_bwd"):
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["C"] = width(4096, 16)
        c["M"] = _log(rng, 1, min(ROWS * 26, ROWS * WIDTH // 2 // c["C"]))
        c.update(post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                 gate=rng.choice(["none", "plain", "sigmoid"]), gate_rows=_log(rng, 1, c["M"]),
                 scale=rng.choice([1.0, 0.5]), beta=rng.random() < 0.5)
        if op == "norm_fwd":
            c["stats"] = rng.random() < 0.5
    elif op == "ckpt":
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["C"] = width(4096)
        c["M"] = _log(rng, 1, ROWS * WIDTH // 2 // c["C"])
        c.update(act=rng.choice(["none", "relu", "gelu", "silu"]), p=rng.choice([0.0, 0.1, 0.5]))
    elif op == "fp4_pack":
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["K"] = width(4096)
        c["M"] = _log(rng, 1, 32768 * WIDTH // 2 // c["K"])
    elif op == "dense_bwd_ckpt":
        c.update(M=_log(rng, 1, ROWS), K=width(WIDTH), N=width(WIDTH), act=rng.choice(["none", "relu", "gelu", "silu"]),
                 p=rng.choice([0.0, 0.1, 0.5]), residual=rng.random() < 0.5)
    else:
        c.update(M=_log(rng, 1, ROWS), K=width(WIDTH), N=width(WIDTH), act=rng.choice(["none", "relu", "gelu", "silu"]),
                 residual=rng.random() < 0.5, refresh=rng.random() < 0.25)
    return c


# ---------------------------------------------------------------------------------------
# Inputs, and the buffers, plans and packed weights that a program keeps.
# ---------------------------------------------------------------------------------------
def _rows(g, m, n, extra, dtype, scale=1.0, shift=0.0, spread=0.0):
    """[m, n] normal values as the first n columns of rows n + extra wide; with `spread`, columns
    of different sizes (activations have outlier columns)."""
    t = torch.randn((m, n + extra), generator=g, device=g.device).mul_(scale)
    if spread:
        t.mul_(torch.exp(spread * torch.randn(n + extra, generator=g, device=g.device)))
    return t.add_(shift).to(DTYPES[dtype])[:, :n]


def _out(m, n, extra, dtype, device):
    return torch.empty((m, n + extra), dtype=DTYPES[dtype], device=device)[:, :n]


def _row_stats(v, kind):
    """[m, 2] fp32: the rows' means (0 where the norm takes none) and reciprocal deviations."""
    if kind == "none":
        return None
    out = torch.empty((v.shape[0], 2), device=v.device)
    step = max(1, (1 << 24) // v.shape[1])
    for a in range(0, v.shape[0], step):
        d = v[a:a + step].double()
        mean = d.mean(1) if kind == "layer" else torch.zeros_like(d[:, 0])
        out[a:a + step, 0] = mean
        out[a:a + step, 1] = ((d - mean[:, None]).square().mean(1) + EPS).rsqrt()
    return out


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    c, op, dt, ex, M = case, case["op"], case["dtype"], case["extra"], case["M"]
    s = dict(case=dict(case), seed=1_000_003 * int(seed) + 54321, offset=int(seed) % 1000)
    if op in ("norm_fwd", "norm_bwd"):
        C, R = c["C"], -(-M // c["gate_rows"])
        vec = lambda base: base + 0.1 * torch.randn(C, generator=g, device=dev)  # noqa: E731
        s["f"] = _rows(g, M, C, ex, dt, 2.0, 0.3)
        s["gate"] = _rows(g, R, C, ex, dt, 0.7, 0.5) if c["gate"] != "none" else None
        s["post_gamma"], s["pre_gamma"] = vec(1.0), vec(1.0)
        s["post_beta"], s["pre_beta"] = (vec(0.0), vec(0.0)) if c["beta"] else (None, None)
        if op == "norm_fwd":
            s["x"] = _rows(g, M, C, ex, dt, 1.0, 0.2)
            s["y"], s["h"] = _out(M, C, ex, dt, dev), _out(M, C, ex, dt, dev)
            s["post_stats"] = torch.empty((M, 2), device=dev) if c["stats"] and c["post"] != "none" else None
            s["pre_stats"] = torch.empty((M, 2), device=dev) if c["stats"] else None
        else:
            # what the forward pass left: y and the rows' statistics
            s["y"] = _rows(g, M, C, ex, dt, 1.5, 0.3)
            s["post_stats"] = _row_stats(s["f"], c["post"])
            s["pre_stats"] = _row_stats(s["y"], c["pre"])
            s["dy"], s["dh"] = _rows(g, M, C, ex, dt), _rows(g, M, C, ex, dt)
            s["dx"], s["df"] = _out(M, C, ex, dt, dev), _out(M, C, ex, dt, dev)
            s["dgate"] = _out(R, C, ex, dt, dev) if c["gate"] != "none" else None
            for k in ("post_gamma", "pre_gamma", "post_beta", "pre_beta"):
                s["d" + k] = torch.empty(C, device=dev) if s[k] is not None else None
        if own:
            import embedding_lookup_feature_amd as elf

            s["norm"] = elf.BlockNorm(C, post=c["post"], pre=c["pre"], post_gamma=s["post_gamma"],
                                      post_beta=s["post_beta"], pre_gamma=s["pre_gamma"], pre_beta=s["pre_beta"],
                                      gate_act="sigmoid" if c["gate"] == "sigmoid" else "none",
                                      gate_rows=c["gate_rows"], scale=c["scale"], eps=EPS)
            if op == "norm_bwd":
                s["workspace"] = torch.empty(max(256, elf.block_norm_bwd_workspace_bytes(s["norm"], M)),
                                             dtype=torch.uint8, device=dev)
        return s
    if op == "ckpt":
        C = c["C"]
        s["x"] = _rows(g, M, C, ex, dt, spread=0.7)
        s["dy"] = _rows(g, M, C, ex, dt)
        s["y"], s["dx"] = _out(M, C, ex, dt, dev), _out(M, C, ex, dt, dev)
        if own:
            import embedding_lookup_feature_amd as elf

            s["ckpt"] = elf.Checkpoint(M, C, dev)
        return s
    K = c["K"]
    if op == "fp4_pack":
        s["x"] = _rows(g, M, K, ex, dt, 1.0 / math.sqrt(K), spread=0.5)
        s["y"] = _out(M, K, ex, dt, dev)
        if own:
            import embedding_lookup_feature_amd as elf

            s["packed"] = elf.Fp4(M, K, dev)
        return s
    N = c["N"]
    s["w"] = _rows(g, N, K, 0, dt, 1.0 / math.sqrt(K))
    s["x"] = _rows(g, M, K, ex, dt, spread=0.7)
    if op == "dense_bwd_ckpt":
        s["pre"] = _rows(g, M, K, 0, dt, spread=0.3)
        s["dz"] = _rows(g, M, N, ex, dt)
        s["dres"] = _rows(g, M, K, ex, dt) if c["residual"] else None
        s["dx"], s["dzb"] = _out(M, K, ex, dt, dev), _out(M, K, ex, dt, dev)
        s["dw"], s["db"] = torch.empty((N, K), device=dev), torch.empty(N, device=dev)
        # the forward pass left its input and its pre-activation in 8 bits
        if own:
            import embedding_lookup_feature_amd as elf

            s["x8"] = elf.ckpt_pack(s["x"], elf.Checkpoint(M, K, dev))
            s["pre8"] = elf.ckpt_pack(s["pre"], elf.Checkpoint(M, K, dev))
            s["workspace"] = torch.empty(max(256, elf.dense_bwd_ckpt_workspace_bytes(M, K, N)), dtype=torch.uint8, device=dev)
        else:
            s["x8"], s["pre8"] = _to8(s["x"].float()), _to8(s["pre"].float())
        del s["x"], s["pre"]
        return s
    s["bias"] = 0.1 * torch.randn(N, generator=g, device=dev)
    s["residual"] = _rows(g, M, N, ex, dt) if c["residual"] else None
    s["y"] = _out(M, N, ex, dt, dev)
    # the weights are packed once, when they are loaded, unless the case packs them in the pass
    if own:
        import embedding_lookup_feature_amd as elf

        s["w4"] = elf.Fp4(N, K, dev)
        if not c["refresh"]:
            elf.fp4_pack(s["w"], s["w4"])
        s["workspace"] = torch.empty(max(256, elf.dense_fwd_fp4_workspace_bytes(M, K, N)), dtype=torch.uint8, device=dev)
    elif not c["refresh"]:
        s["w4"] = _to4(s["w"].float())
    if not c["refresh"]:
        del s["w"]
    return s


# ---------------------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------------------
_LOW = 0xFFFFFFFF


def _micro(v, top, low, bits):
    """fp32 [m, n] rounded to blocks of 32 with numbers of `bits` fraction bits, largest `top`,
    smallest binary exponent `low`; every step but the rounding is exact."""
    m, n = v.shape
    pad = -n % BLOCK
    b = torch.nn.functional.pad(v, (0, pad)).view(m, -1, BLOCK)
    frac, e = torch.frexp(b.abs().amax(-1, keepdim=True))  # amax = frac 2^e, frac in [0.5, 1)
    tf, te = math.frexp(top)
    e = torch.where(frac > tf, e - te + 1, e - te).clamp(min=-126)
    one = torch.ones((), device=v.device)
    b = b * torch.ldexp(one, -e)
    _, k = torch.frexp(b)
    step = torch.ldexp(one, torch.clamp(k - 1, min=low) - bits)
    b = torch.round(b / step) * step  # ties to even
    return (b * torch.ldexp(one, e)).view(m, -1)[:, :n]


def _to8(v):
    return _micro(v, 448.0, -6, 3)


def _to4(v):
    return _micro(v, 6.0, 0, 1)


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
    return bits >= t, 65536.0 / (65536 - t)


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


def _plain_gate(s):
    c = s["case"]
    if s["gate"] is None:
        return 1.0, None
    u = s["gate"].float()
    gate = 1.0 / (1.0 + torch.exp(-u)) if c["gate"] == "sigmoid" else u
    return gate[torch.arange(c["M"], device=u.device) // c["gate_rows"]], gate


def _plain_norm(v, kind):
    """(normalised rows, [m, 2] of mean and rstd)."""
    if kind == "none":
        return v, None
    mean = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, :1])
    d = v - mean
    rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / v.shape[1] + EPS)
    return d * rstd, torch.cat([mean, rstd], 1)


def _plain_norm_fwd(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    zero = torch.zeros((), device=s["x"].device)
    post_beta = s["post_beta"] if s["post_beta"] is not None else zero
    pre_beta = s["pre_beta"] if s["pre_beta"] is not None else zero
    fh, post_stats = _plain_norm(s["f"].float(), c["post"])
    y = s["x"].float() + c["scale"] * _plain_gate(s)[0] * (fh * s["post_gamma"] + post_beta)
    yh, pre_stats = _plain_norm(y, c["pre"])
    out = {"y": y.to(dt), "h": (yh * s["pre_gamma"] + pre_beta).to(dt)}
    if c["stats"]:
        out["pre_stats"] = pre_stats
        if c["post"] != "none":
            out["post_stats"] = post_stats
    return out


def _plain_norm_grad(d, vh, stats, kind):
    """Gradient at the norm's input from the one at its output."""
    if kind == "none":
        return d
    n = d.shape[1]
    g = d - vh * ((d * vh).sum(1, keepdim=True) / n)
    if kind == "layer":
        g = g - d.sum(1, keepdim=True) / n
    return g * stats[:, 1:]


def _plain_norm_bwd(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    M, C, S = c["M"], c["C"], c["gate_rows"]
    g, gate = _plain_gate(s)
    yh = (s["y"].float() - s["pre_stats"][:, :1]) * s["pre_stats"][:, 1:]
    fh = s["f"].float()
    if c["post"] != "none":
        fh = (fh - s["post_stats"][:, :1]) * s["post_stats"][:, 1:]
    dh = s["dh"].float()
    out = {"dpre_gamma": (dh * yh).sum(0)}
    if c["beta"]:
        out["dpre_beta"] = dh.sum(0)
    D = s["dy"].float() + _plain_norm_grad(dh * s["pre_gamma"], yh, s["pre_stats"], c["pre"])
    out["dx"] = D.to(dt)
    if gate is not None:
        t = fh * s["post_gamma"]
        if c["beta"]:
            t = t + s["post_beta"]
        dg = torch.nn.functional.pad(c["scale"] * D * t, (0, 0, 0, -M % S)).view(-1, S, C).sum(1)
        if c["gate"] == "sigmoid":
            dg = dg * gate * (1.0 - gate)
        out["dgate"] = dg.to(dt)
    d_t = c["scale"] * g * D
    out["dpost_gamma"] = (d_t * fh).sum(0)
    if c["beta"]:
        out["dpost_beta"] = d_t.sum(0)
    out["df"] = _plain_norm_grad(d_t * s["post_gamma"], fh, s["post_stats"], c["post"]).to(dt)
    return out


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    dt = DTYPES[c["dtype"]]
    if op == "ckpt":
        u = _to8(s["x"].float())
        return {"y": _drop(_act(u, c["act"]), s).to(dt), "dx": _drop(s["dy"].float() * _act_grad(u, c["act"]), s).to(dt)}
    if op == "fp4_pack":
        return {"y": _to4(s["x"].float()).to(dt)}
    if op == "dense_bwd_ckpt":
        dz = s["dz"].float()
        dx = dz @ s["w"].float()
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        dzb = _drop(dx * _act_grad(s["pre8"], c["act"]), s)
        return {"dx": dx.to(dt), "dzb": dzb.to(dt), "dw": dz.t() @ s["x8"], "db": dz.sum(0)}
    w = _to4(s["w"].float()) if c["refresh"] else s["w4"]
    y = _act(_to4(s["x"].float()) @ w.t() + s["bias"], c["act"])
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return {"y": y.to(dt)}


# ---------------------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------------------
def _own(s):
    import embedding_lookup_feature_amd as elf

    c, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        elf.block_norm_fwd(s["norm"], s["x"], s["y"], s["h"], f=s["f"], gate=s["gate"], post_stats=s["post_stats"],
                           pre_stats=s["pre_stats"])
        return {k: s[k] for k in ("y", "h", "post_stats", "pre_stats") if s[k] is not None}
    if op == "norm_bwd":
        elf.block_norm_bwd(s["norm"], s["y"], s["dx"], dy=s["dy"], dh=s["dh"], f=s["f"], gate=s["gate"], df=s["df"],
                           dgate=s["dgate"], post_stats=s["post_stats"], pre_stats=s["pre_stats"],
                           dpost_gamma=s["dpost_gamma"], dpost_beta=s["dpost_beta"], dpre_gamma=s["dpre_gamma"],
                           dpre_beta=s["dpre_beta"], workspace=s["workspace"])
        return {k: s[k] for k in ("dx", "df", "dgate", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")
                if s[k] is not None}
    drop = elf.Dropout(c["p"], s["seed"], s["offset"]) if c.get("p", 0.0) > 0.0 else None
    if op == "ckpt":
        elf.ckpt_pack(s["x"], s["ckpt"])
        elf.ckpt_act_dropout_fwd(s["ckpt"], s["y"], act=c["act"], dropout=drop)
        elf.ckpt_act_dropout_bwd(s["dy"], s["ckpt"], s["dx"], act=c["act"], dropout=drop)
        return {"y": s["y"], "dx": s["dx"]}
    if op == "fp4_pack":
        return {"y": elf.fp4_unpack(elf.fp4_pack(s["x"], s["packed"]), s["y"])}
    if op == "dense_bwd_ckpt":
        elf.dense_bwd_ckpt(s["x8"], s["w"], s["dz"], s["dw"], s["db"], dx=s["dx"], dres=s["dres"], dzb=s["dzb"],
                           pre=s["pre8"], act=c["act"], dropout=drop, workspace=s["workspace"])
        return {k: s[k] for k in ("dx", "dzb", "dw", "db")}
    if c["refresh"]:
        elf.fp4_pack(s["w"], s["w4"])
    elf.dense_fwd_fp4(s["x"], s["w4"], s["bias"], s["y"], act=c["act"], residual=s["residual"], workspace=s["workspace"])
    return {"y": s["y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------------------
def work(case):
    c, op, e, M = case, case["op"], SIZE[case["dtype"]], case["M"]
    if op in ("norm_fwd", "norm_bwd"):
        C = c["C"]
        n, g = M * C, -(-M // c["gate_rows"]) * C if c["gate"] != "none" else 0
        vec = 4 * C * (4 if c["beta"] else 2)
        stats = 8 * M * (2 if c["post"] != "none" else 1)
        if op == "norm_fwd":  # x, f, gate -> y, h
            return {"bytes": e * (4 * n + g) + vec + (stats if c["stats"] else 0), "flops": 14 * n}
        return {"bytes": e * (6 * n + 2 * g) + 2 * vec + stats, "flops": 40 * n}  # dy, dh, y, f, gate -> dx, df, dgate
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if op == "ckpt":  # x stored and recomputed from, dy -> y, dx; the 8 bits written and read once
        n, q = M * c["C"], M * (c["C"] + blocks(c["C"]))
        return {"bytes": e * 4 * n + 2 * q, "flops": 30 * n}
    K = c["K"]
    if op == "fp4_pack":
        n, q = M * K, M * (K // 2 + blocks(K))
        return {"bytes": e * 2 * n + 2 * q, "flops": 10 * n}
    N = c["N"]
    if op == "dense_bwd_ckpt":
        q = M * (K + blocks(K))
        b = e * (M * K * (2 + int(c["residual"])) + N * K + M * N) + 2 * q + 4 * (N * K + N)
        return {"bytes": b, "flops": 4 * M * K * N}
    b = e * (M * K + M * N * (1 + int(c["residual"]))) + (e * N * K if c["refresh"] else N * (K // 2 + blocks(K))) + 4 * N
    return {"bytes": b, "flops": 2 * M * K * N}


# ---------------------------------------------------------------------------------------
# The operators' definition in 64 bits, apart from the forms above.
# ---------------------------------------------------------------------------------------
def _numbers(exp_bits, frac_bits, count):
    """The first `count` magnitudes of a small float format, by their codes."""
    bias, out = 2 ** (exp_bits - 1) - 1, []
    for code in range(count):
        ex, fr = code >> frac_bits, code & ((1 << frac_bits) - 1)
        out.append((fr / 2**frac_bits) * 2.0 ** (1 - bias) if ex == 0 else (1 + fr / 2**frac_bits) * 2.0 ** (ex - bias))
    return out


def _exact_micro(v, numbers):
    """float64 [m, n]: every value replaced by its block's nearest number (even codes at ties)."""
    table = torch.tensor(numbers, dtype=torch.float64, device=v.device)
    mid = (table[1:] + table[:-1]) / 2
    m, n = v.shape
    out = torch.empty_like(v)
    for j in range(0, n, BLOCK):
        b = v[:, j:j + BLOCK]
        amax = b.abs().max(dim=1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.clamp(amax / numbers[-1], min=2.0**-126)))
        # the logarithm is rounded: settle the power by comparisons
        e = torch.where(amax > numbers[-1] * torch.exp2(e), e + 1, e)
        e = torch.where((e > -126) & (amax <= numbers[-1] * torch.exp2(e - 1)), e - 1, e)
        w = torch.exp2(e)
        q = (b / w).abs()
        i = torch.bucketize(q, mid)  # numbers of midpoints below
        i = i + ((i < mid.numel()) & (i % 2 == 1) & (q == mid[i.clamp(max=mid.numel() - 1)])).long()
        out[:, j:j + BLOCK] = torch.where(b < 0, -table[i], table[i]) * w
    return out


_E4M3, _E2M1 = _numbers(4, 3, 127), _numbers(2, 1, 8)


def _exact_mask(m, n, p, seed, offset):
    """[m, n] factors (0 or the scale) of the dropout mask, by numpy's unsigned integers."""
    t = int(math.floor(65536 * p + 0.5))
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
    return torch.from_numpy(np.where(bits >= t, 65536.0 / (65536 - t), 0.0))


def _exact_act(u, act, grad=False):
    if act == "none":
        return torch.ones_like(u) if grad else u
    if act == "relu":
        return torch.heaviside(u, torch.zeros_like(u)) if grad else torch.clamp(u, min=0.0)
    if act == "gelu":  # u Phi(u); Phi(u) + u phi(u)
        phi = torch.special.ndtr(u)
        return phi + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi) if grad else u * phi
    sig = torch.sigmoid(u)
    return sig + u * sig * (1 - sig) if grad else u * sig


def _exact_norm(s):
    c = s["case"]
    M, C, S, back = c["M"], c["C"], c["gate_rows"], c["op"] == "norm_bwd"
    dev = s["f"].device
    out = {k: torch.empty((M, C), dtype=torch.float64) for k in (("dx", "df") if back else ("y", "h"))}
    if not back and c["stats"]:
        out["pre_stats"] = torch.empty((M, 2), dtype=torch.float64)
        if c["post"] != "none":
            out["post_stats"] = torch.empty((M, 2), dtype=torch.float64)
    vec = lambda k, d: s[k].double() if s[k] is not None else torch.full((C,), d, dtype=torch.float64, device=dev)  # noqa: E731
    ga, ba, gb, bb = vec("post_gamma", 1), vec("post_beta", 0), vec("pre_gamma", 1), vec("pre_beta", 0)
    sums = {k: torch.zeros(C, dtype=torch.float64, device=dev) for k in ("post_gamma", "post_beta", "pre_gamma", "pre_beta")}
    dgate = torch.zeros((-(-M // S), C), dtype=torch.float64, device=dev)
    step = max(1, (1 << 23) // C)

    def moments(v, kind, name, a, b):
        if kind == "none":
            return 0.0, 1.0
        if back:
            st = s[name][a:b].double()
            return st[:, :1], st[:, 1:]
        mu = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
        r = ((v.var(1, unbiased=False, keepdim=True) if kind == "layer" else (v * v).mean(1, keepdim=True)) + EPS) ** -0.5
        if c["stats"]:
            out[name][a:b] = torch.cat([mu, r], 1).cpu()
        return mu, r

    def pull(g, vh, r, kind):
        if kind == "none":
            return g
        w = (g * vh).mean(1, keepdim=True) * vh
        return r * ((g - g.mean(1, keepdim=True) if kind == "layer" else g) - w)

    for a in range(0, M, step):
        b = min(M, a + step)
        f = s["f"][a:b].double()
        rows = torch.arange(a, b, device=dev) // S
        mu, fr = moments(f, c["post"], "post_stats", a, b)
        fh = (f - mu) * fr
        t = ga * fh + ba
        raw = s["gate"][rows].double() if s["gate"] is not None else torch.ones_like(t)
        g = torch.sigmoid(raw) if c["gate"] == "sigmoid" else raw
        y = s["y"][a:b].double() if back else s["x"][a:b].double() + c["scale"] * (g * t)
        mu, yr = moments(y, c["pre"], "pre_stats", a, b)
        yh = (y - mu) * yr
        if not back:
            out["y"][a:b], out["h"][a:b] = y.cpu(), (gb * yh + bb).cpu()
            continue
        dh = s["dh"][a:b].double()
        D = s["dy"][a:b].double() + pull(gb * dh, yh, yr, c["pre"])
        du = D * g * c["scale"]
        for k, v in (("pre_gamma", dh * yh), ("pre_beta", dh), ("post_gamma", du * fh), ("post_beta", du)):
            sums[k] += v.sum(0)
        dg = D * t * c["scale"]
        dgate.index_add_(0, rows, dg * g * (1 - g) if c["gate"] == "sigmoid" else dg)
        out["dx"][a:b], out["df"][a:b] = D.cpu(), pull(ga * du, fh, fr, c["post"]).cpu()
    if back:
        if s["gate"] is not None:
            out["dgate"] = dgate.cpu()
        out.update({"d" + k: v.cpu() for k, v in sums.items() if s[k] is not None})
    return out


def exact(case, seed):
    global own
    c, op = case, case["op"]
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s)
    wide = lambda k: s[k].double()  # noqa: E731
    if op == "fp4_pack":
        return {"y": _exact_micro(wide("x"), _E2M1).cpu()}
    if op == "dense_fp4":
        w = _exact_micro(wide("w"), _E2M1) if c["refresh"] else s["w4"].double()
        z = torch.mm(_exact_micro(wide("x"), _E2M1), w.t().contiguous()) + wide("bias")
        y = _exact_act(z, c["act"])
        return {"y": (y if s["residual"] is None else y + wide("residual")).cpu()}
    n = c["C"] if op == "ckpt" else c["K"]
    mask = _exact_mask(c["M"], n, c["p"], s["seed"], s["offset"]).to(s["w" if op != "ckpt" else "x"].device) if c["p"] > 0 else None
    pick = lambda v: v if mask is None else torch.where(mask > 0, v * mask, torch.zeros_like(v))  # noqa: E731
    if op == "ckpt":
        u = _exact_micro(wide("x"), _E4M3)
        return {"y": pick(_exact_act(u, c["act"])).cpu(), "dx": pick(wide("dy") * _exact_act(u, c["act"], True)).cpu()}
    dx = torch.mm(wide("dz"), wide("w"))
    if s["dres"] is not None:
        dx = dx + wide("dres")
    dzb = pick(dx * _exact_act(s["pre8"].double(), c["act"], True))
    dw = torch.mm(wide("dz").t().contiguous(), s["x8"].double())
    return {"dx": dx.cpu(), "dzb": dzb.cpu(), "dw": dw.cpu(), "db": wide("dz").sum(0).cpu()}

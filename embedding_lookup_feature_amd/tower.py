"""Python binding of the dense-tower operators (the C ABI in ``include/embtower.h``).

Argument marshalling only, in the manner of ``embcore``: torch tensors are passed as device
pointers plus sizes and row strides, on torch's current HIP stream unless a stream is given;
outputs and workspaces belong to the caller (a workspace that is not given is allocated here
for the call, on the call's stream).  Two-dimensional operands may be row-strided views (last
dimension dense).
"""
import ctypes
import os
import re

import torch

from . import embcore as ec

HEADER = os.path.join(os.path.dirname(ec.HERE), "include", "embtower.h")

EL_ACT_GELU, EL_ACT_SILU = 2, 3
ACTIVATIONS = {"none": ec.EL_ACT_NONE, "relu": ec.EL_ACT_RELU, "gelu": EL_ACT_GELU, "silu": EL_ACT_SILU}


class ElDropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step", ctypes.c_void_p)]


class Dropout:
    """The mask of one dropout: keep probability 1 - p, drawn from (seed, offset, row, column).
    `step`, an int64 device tensor of one element, is added to the offset when the work runs, so
    that the replays of a captured graph draw other masks."""

    def __init__(self, p: float, seed: int, offset: int = 0, step: torch.Tensor = None):
        if step is not None and (step.dtype != torch.int64 or step.numel() != 1):
            raise ValueError("step must be an int64 tensor of one element")
        self.step = step
        self.c = ElDropout(float(p), int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                           ec._dev(step, "step") if step is not None else None)


_bound = None


def lib() -> ctypes.CDLL:
    """The loaded library with this header's functions declared."""
    global _bound
    if _bound is None:
        L = ec.lib()
        vp, i32, i64, u32, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                      ctypes.c_float, ctypes.c_size_t)
        dt, D = ctypes.c_int, ctypes.POINTER(ElDropout)
        L.el_act_dropout_fwd.argtypes = [vp, i64, vp, i64, i32, i32, u32, D, vp, i64, dt, vp]
        L.el_act_dropout_bwd.argtypes = [vp, i64, vp, i64, i32, i32, u32, D, vp, i64, dt, vp]
        L.el_dense_fwd.argtypes = [vp, i64, i32, i32, vp, vp, i32, u32, D, vp, i64, vp, i64, vp, i64, dt, vp, sz, vp]
        L.el_dense_bwd.argtypes = [vp, i64, i32, i32, vp, i32, vp, i64, vp, i64, vp, i64, u32, D, vp, i64, vp, i64,
                                   vp, vp, dt, vp, sz, vp]
        L.el_group_norm_fwd.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, f32, u32, vp, i64, vp, vp, dt, vp,
                                        sz, vp]
        L.el_group_norm_bwd.argtypes = [vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, u32, vp, i64, vp,
                                        vp, dt, vp, sz, vp]
        for name in ("el_act_dropout_fwd", "el_act_dropout_bwd", "el_dense_fwd", "el_dense_bwd",
                     "el_group_norm_fwd", "el_group_norm_bwd"):
            getattr(L, name).restype = ctypes.c_int
        for name, n in (("el_dense_fwd_workspace_bytes", 3), ("el_dense_bwd_workspace_bytes", 3),
                        ("el_group_norm_fwd_workspace_bytes", 4), ("el_group_norm_bwd_workspace_bytes", 4)):
            getattr(L, name).argtypes = [i32] * n
            getattr(L, name).restype = sz
        _bound = L
    return _bound


def header_functions():
    """Names of the functions `include/embtower.h` declares."""
    text = open(HEADER).read()
    return re.findall(r"EL_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


def _act(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _drop(dropout):
    return ctypes.byref(dropout.c) if dropout is not None else None


def _mat(t: torch.Tensor, name: str, shape, dtype):
    """(pointer, row stride) of a row-strided [rows, cols] operand; (None, cols) of None."""
    if t is None:
        return None, shape[1]
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    ld, cs = t.stride()
    if cs != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    # the row stride of one row (or none) says nothing
    return t.data_ptr(), ld if shape[0] > 1 else max(ld, shape[1])


def _stream(stream, t: torch.Tensor):
    """The stream's handle; without one, torch's current stream on t's device (its raw handle:
    a Stream object costs more than the rest of a small call's marshalling)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.device.index)
    return ec._stream(stream)


def _vec(t: torch.Tensor, name: str, n: int, dtype=torch.float32):
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n:
        raise ValueError(f"{name} must hold {n} values of {dtype}")
    return ec._dev(t, name)


def _rows_cols(t: torch.Tensor, name: str):
    s = t.shape
    if len(s) != 2:
        raise ValueError(f"{name} must be 2-D")
    return s


def _too_large(*n: int):
    """The ABI takes sizes in 32 bits, and ctypes would cut larger ones without a word."""
    raise ValueError(f"sizes must be below 2^31, got {list(n)}")


def _workspace(ws, need: int, device, stream):
    if ws is None and need > 0:
        ws = ec._scratch(need, device, stream)
    if ws is None:
        return None, 0, None
    return ec._dev(ws, "workspace"), ws.numel() * ws.element_size(), ws


def act_dropout_fwd(x: torch.Tensor, y: torch.Tensor, act: str = "none", dropout: Dropout = None,
                    residual: torch.Tensor = None, stream=None):
    """y = residual + drop(act(x)); x, y, residual [M, N] of one dtype (fp32, fp16, bf16)."""
    shape = M, N = _rows_cols(x, "x")
    if (M | N) >> 31:
        _too_large(M, N)
    xp, ldx = _mat(x, "x", shape, x.dtype)
    rp, ldr = _mat(residual, "residual", shape, x.dtype)
    yp, ldy = _mat(y, "y", shape, x.dtype)
    ec._check(lib().el_act_dropout_fwd(xp, ldx, rp, ldr, M, N, _act(act), _drop(dropout), yp, ldy,
                                       ec._dtype(x, "x"), _stream(stream, x)))
    return y


def act_dropout_bwd(dy: torch.Tensor, x: torch.Tensor, dx: torch.Tensor, act: str = "none",
                    dropout: Dropout = None, stream=None):
    """dx = drop(dy * act'(x)), the mask of the forward with the same dropout (x may be None
    with act "none")."""
    shape = M, N = _rows_cols(dy, "dy")
    if (M | N) >> 31:
        _too_large(M, N)
    dp, lddy = _mat(dy, "dy", shape, dy.dtype)
    xp, ldx = _mat(x, "x", shape, dy.dtype)
    op, lddx = _mat(dx, "dx", shape, dy.dtype)
    ec._check(lib().el_act_dropout_bwd(dp, lddy, xp, ldx, M, N, _act(act), _drop(dropout), op, lddx,
                                       ec._dtype(dy, "dy"), _stream(stream, dy)))
    return dx


def dense_fwd_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().el_dense_fwd_workspace_bytes(M, K, N))


def dense_bwd_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().el_dense_bwd_workspace_bytes(M, K, N))


def dense_fwd(x: torch.Tensor, w: torch.Tensor, bias, y: torch.Tensor, act: str = "none",
              dropout: Dropout = None, residual: torch.Tensor = None, pre: torch.Tensor = None,
              workspace: torch.Tensor = None, stream=None):
    """z = x @ w.T + bias; y = residual + drop(act(z)); pre (when given) = z.  x [M, K], w [N, K]
    contiguous, bias fp32 [N] or None, y / residual / pre [M, N], bf16 or fp16."""
    M, K = _rows_cols(x, "x")
    N = _rows_cols(w, "w")[0]
    if (M | K | N) >> 31:
        _too_large(M, K, N)
    if w.shape != (N, K) or w.dtype is not x.dtype:
        raise ValueError(f"w must be [N, {K}] of {x.dtype}")
    xp, ldx = _mat(x, "x", (M, K), x.dtype)
    rp, ldr = _mat(residual, "residual", (M, N), x.dtype)
    pp, ldp = _mat(pre, "pre", (M, N), x.dtype)
    yp, ldy = _mat(y, "y", (M, N), x.dtype)
    wsp, wsn, keep = _workspace(workspace, 0 if workspace is not None else dense_fwd_workspace_bytes(M, K, N),
                                x.device, stream)
    ec._check(lib().el_dense_fwd(xp, ldx, M, K, ec._dev(w, "w"), _vec(bias, "bias", N), N, _act(act), _drop(dropout),
                                 rp, ldr, pp, ldp, yp, ldy, ec._dtype(x, "x"), wsp, wsn, _stream(stream, x)))
    return y


def dense_bwd(x: torch.Tensor, w: torch.Tensor, dz: torch.Tensor, dw: torch.Tensor, db: torch.Tensor = None,
              dx: torch.Tensor = None, dres: torch.Tensor = None, dzb: torch.Tensor = None,
              pre: torch.Tensor = None, act: str = "none", dropout: Dropout = None,
              workspace: torch.Tensor = None, stream=None):
    """dw = dz.T @ x, db = dz.sum(0) (fp32); dx = dz @ w + dres; dzb = drop(dx * act'(pre)), the
    dz of the layer below (act, dropout and pre are that layer's).  dx, dres, dzb, pre [M, K]."""
    M, K = _rows_cols(x, "x")
    N = _rows_cols(w, "w")[0]
    if (M | K | N) >> 31:
        _too_large(M, K, N)
    if w.shape != (N, K) or w.dtype is not x.dtype:
        raise ValueError(f"w must be [N, {K}] of {x.dtype}")
    xp, ldx = _mat(x, "x", (M, K), x.dtype)
    zp, ldz = _mat(dz, "dz", (M, N), x.dtype)
    dxp, lddx = _mat(dx, "dx", (M, K), x.dtype)
    rp, ldr = _mat(dres, "dres", (M, K), x.dtype)
    bp, ldb = _mat(dzb, "dzb", (M, K), x.dtype)
    pp, ldp = _mat(pre, "pre", (M, K), x.dtype)
    wsp, wsn, keep = _workspace(workspace, 0 if workspace is not None else dense_bwd_workspace_bytes(M, K, N),
                                x.device, stream)
    if dw.numel() != N * K:
        raise ValueError(f"dw must be [{N}, {K}]")
    ec._check(lib().el_dense_bwd(xp, ldx, M, K, ec._dev(w, "w"), N, zp, ldz, rp, ldr, dxp, lddx, _act(act),
                                 _drop(dropout), pp, ldp, bp, ldb, _vec(dw, "dw", N * K), _vec(db, "db", N),
                                 ec._dtype(x, "x"), wsp, wsn, _stream(stream, x)))
    return dx, dw, db


def group_norm_fwd_workspace_bytes(B: int, S: int, C: int, G: int) -> int:
    return int(lib().el_group_norm_fwd_workspace_bytes(B, S, C, G))


def group_norm_bwd_workspace_bytes(B: int, S: int, C: int, G: int) -> int:
    return int(lib().el_group_norm_bwd_workspace_bytes(B, S, C, G))


def _samples(x: torch.Tensor, positions: int, groups: int):
    rows, C = _rows_cols(x, "x")
    S = int(positions)
    if S < 1 or rows % S != 0:
        raise ValueError(f"x must have a whole number of samples of {S} rows, got {rows}")
    B, G = rows // S, int(groups)
    if (B | S | C | G) >> 31 > 0:  # (a negative G is refused as such)
        _too_large(B, S, C, G)
    return B, S, C, G


def group_norm_fwd(x: torch.Tensor, gamma, beta, y: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   positions: int, groups: int, eps: float = 1e-5, act: str = "none", lengths=None,
                   workspace: torch.Tensor = None, stream=None):
    """y = act(gamma (x - mean) rstd + beta) over groups of channels, x [B * positions, C]
    (channels last); mean, rstd fp32 [B, groups] are written; lengths: int32 [B] valid positions
    or None; padded positions of y are zero."""
    B, S, C, G = _samples(x, positions, groups)
    xp, ldx = _mat(x, "x", x.shape, x.dtype)
    yp, ldy = _mat(y, "y", x.shape, x.dtype)
    wsp, wsn, keep = _workspace(workspace, 0 if workspace is not None else group_norm_fwd_workspace_bytes(B, S, C, G),
                                x.device, stream)
    ec._check(lib().el_group_norm_fwd(xp, ldx, B, S, C, G, _vec(lengths, "lengths", B, torch.int32),
                                      _vec(gamma, "gamma", C), _vec(beta, "beta", C), float(eps), _act(act), yp, ldy,
                                      _vec(mean, "mean", B * G), _vec(rstd, "rstd", B * G), ec._dtype(x, "x"), wsp,
                                      wsn, _stream(stream, x)))
    return y


def group_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma, beta, mean: torch.Tensor, rstd: torch.Tensor,
                   dx: torch.Tensor, dgamma, dbeta, positions: int, groups: int, act: str = "none", lengths=None,
                   workspace: torch.Tensor = None, stream=None):
    """Gradients of group_norm_fwd from its inputs and its mean / rstd: dx (zero at padded
    positions), dgamma and dbeta (fp32 [C], either may be None)."""
    B, S, C, G = _samples(x, positions, groups)
    dp, lddy = _mat(dy, "dy", x.shape, x.dtype)
    xp, ldx = _mat(x, "x", x.shape, x.dtype)
    op, lddx = _mat(dx, "dx", x.shape, x.dtype)
    wsp, wsn, keep = _workspace(workspace, 0 if workspace is not None else group_norm_bwd_workspace_bytes(B, S, C, G),
                                x.device, stream)
    ec._check(lib().el_group_norm_bwd(dp, lddy, xp, ldx, B, S, C, G, _vec(lengths, "lengths", B, torch.int32),
                                      _vec(gamma, "gamma", C), _vec(beta, "beta", C), _vec(mean, "mean", B * G),
                                      _vec(rstd, "rstd", B * G), _act(act), op, lddx, _vec(dgamma, "dgamma", C),
                                      _vec(dbeta, "dbeta", C), ec._dtype(x, "x"), wsp, wsn, _stream(stream, x)))
    return dx, dgamma, dbeta

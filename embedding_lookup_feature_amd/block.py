"""Python binding of the residual block's operators (the C ABI in ``include/embblock.h``).

Argument marshalling only, in the manner of ``tower``: torch tensors are passed as device
pointers plus sizes and row strides, on torch's current HIP stream unless a stream is given, with
the operands' device made current for the call; outputs and workspaces belong to the caller (a
workspace that is not given is allocated here for the call, on the call's stream).
Two-dimensional operands may be row-strided views (last dimension dense).
"""
import ctypes
import os
import re

import torch

from . import embcore as ec
from . import tower as tw

HEADER = os.path.join(os.path.dirname(ec.HERE), "include", "embblock.h")

NORMS = {"none": 0, "rms": 1, "layer": 2}
GATES = {"none": 0, "sigmoid": 1}
MICRO_BLOCK = 32
PARAMS = ("post_gamma", "post_beta", "pre_gamma", "pre_beta")


class ElBlockNorm(ctypes.Structure):
    _fields_ = [("post", ctypes.c_uint32), ("pre", ctypes.c_uint32), ("gate_act", ctypes.c_uint32),
                ("gate_rows", ctypes.c_int32), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("post_gamma", ctypes.c_void_p), ("post_beta", ctypes.c_void_p),
                ("pre_gamma", ctypes.c_void_p), ("pre_beta", ctypes.c_void_p)]


_bound = None


def lib() -> ctypes.CDLL:
    """The loaded library with this header's functions declared."""
    global _bound
    if _bound is None:
        L = ec.lib()
        vp, i32, i64, u32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t)
        dt, D, P = ctypes.c_int, ctypes.POINTER(tw.ElDropout), ctypes.POINTER(ElBlockNorm)
        L.el_block_norm_fwd.argtypes = [P, vp, i64, vp, i64, vp, i64, i32, i32, vp, i64, vp, i64, vp, vp, dt, vp]
        L.el_block_norm_bwd.argtypes = [P, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, vp, vp, vp, i64, vp,
                                        i64, vp, i64, vp, vp, vp, vp, dt, vp, sz, vp]
        L.el_ckpt_pack.argtypes = [vp, i64, i32, i32, dt, vp, vp, vp]
        L.el_ckpt_act_dropout_fwd.argtypes = [vp, vp, i32, i32, u32, D, vp, i64, dt, vp]
        L.el_ckpt_act_dropout_bwd.argtypes = [vp, i64, vp, vp, i32, i32, u32, D, vp, i64, dt, vp]
        L.el_dense_bwd_ckpt.argtypes = [vp, vp, i32, i32, vp, i32, vp, i64, vp, i64, vp, i64, u32, D, vp, vp, vp, i64,
                                        vp, vp, dt, vp, sz, vp]
        L.el_fp4_pack.argtypes = [vp, i64, i32, i32, dt, vp, vp, vp]
        L.el_fp4_unpack.argtypes = [vp, vp, i32, i32, vp, i64, dt, vp]
        L.el_dense_fwd_fp4.argtypes = [vp, i64, i32, i32, vp, vp, vp, i32, u32, vp, i64, vp, i64, dt, vp, sz, vp]
        for name in header_functions():
            getattr(L, name).restype = ctypes.c_int
        for name in ("el_block_norm_bwd_workspace_bytes", "el_dense_bwd_ckpt_workspace_bytes",
                     "el_dense_fwd_fp4_workspace_bytes"):
            getattr(L, name).argtypes = [i32] * 3
            getattr(L, name).restype = sz
        _bound = L
    return _bound


def header_functions():
    """Names of the functions `include/embblock.h` declares."""
    text = open(HEADER).read()
    return re.findall(r"EL_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


_current_device = torch._C._cuda_getDevice


def _device(t: torch.Tensor, name: str) -> int:
    """The index of t's device; t must be on one."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a device tensor")
    return i


def _launch(fn, dev: int, stream, *args):
    """Calls fn(*args, stream) with the operands' device current (the default stream's handle names
    none); without a stream, on torch's current one there."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else ec._stream(stream)
    if dev == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status:
        ec._check(status)


def _mat(t, name: str, shape, dtype, dev: int):
    """(pointer, row stride) of a row-strided [rows, cols] operand on device dev; (None, cols) of None."""
    if t is None:
        return None, shape[1]
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {list(shape)} of {dtype} on device {dev}, got {list(t.shape)} of {t.dtype} on "
                         f"{t.device}")
    ld, cs = t.stride()
    if cs != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    # the row stride of one row (or none) says nothing
    return t.data_ptr(), ld if shape[0] > 1 else max(ld, shape[1])


def _vec(t, name: str, n: int, dev: int):
    """The pointer of n contiguous fp32 values."""
    if t is None:
        return None
    if t.numel() != n or t.dtype is not torch.float32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous values of float32 on device {dev}")
    return t.data_ptr()


def _drop(dropout, dev: int):
    if dropout is not None and dropout.step is not None and dropout.step.get_device() != dev:
        raise ValueError(f"the dropout's step must be on device {dev}, got {dropout.step.device}")
    return tw._drop(dropout)


def _workspace(ws, need, like: torch.Tensor, dev: int, stream):
    """(pointer, bytes, the tensor that holds them); `need` is asked where none is given."""
    if ws is None:
        n = need()
        if n == 0:
            return None, 0, None
        ws = ec._scratch(n, like.device, stream)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous on device {dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


class BlockNorm:
    """The parameters around one residual block of C columns: the norms `post` behind it ("none",
    "rms", "layer") and `pre` before the next ("rms", "layer") with their gammas and betas (fp32 [C]
    or None), the gate's activation ("none", "sigmoid"), the number of consecutive rows that share
    one row of the gate, and the residual scale.  Calls read the tensors where they lie then: one whose
    storage was replaced (same size, type and device) is followed."""

    def __init__(self, C: int, post: str = "none", pre: str = "rms", post_gamma: torch.Tensor = None,
                 post_beta: torch.Tensor = None, pre_gamma: torch.Tensor = None, pre_beta: torch.Tensor = None,
                 gate_act: str = "none", gate_rows: int = 1, scale: float = 1.0, eps: float = 1e-5):
        if post not in NORMS:
            raise ValueError(f"post must be one of {sorted(NORMS)}, got {post!r}")
        if pre not in NORMS or pre == "none":
            raise ValueError(f"pre must be \"rms\" or \"layer\", got {pre!r}")
        if gate_act not in GATES:
            raise ValueError(f"gate_act must be one of {sorted(GATES)}, got {gate_act!r}")
        if not 1 <= gate_rows < 2**31:
            raise ValueError(f"gate_rows must be from 1 to 2^31 - 1, got {gate_rows}")
        if not 1 <= C < 2**31:
            raise ValueError(f"C must be from 1 to 2^31 - 1, got {C}")
        self.C, self.gate_rows = int(C), int(gate_rows)
        self.params = (post_gamma, post_beta, pre_gamma, pre_beta)
        self.device = next((_device(p, name) for p, name in zip(self.params, PARAMS) if p is not None), None)
        for p, name in zip(self.params, PARAMS):
            if p is not None and p.get_device() != self.device:
                raise ValueError(f"{name} must be on the other parameters' device")
        self._plain = NORMS[post], NORMS[pre], GATES[gate_act], self.gate_rows, float(scale), float(eps)
        self._bind()

    def _bind(self):
        ptrs = [_vec(p, name, self.C, self.device) for p, name in zip(self.params, PARAMS)]
        self._ref = ctypes.byref(ElBlockNorm(*self._plain, *ptrs))
        self._held = [(p, p.data_ptr(), p.numel()) for p in self.params if p is not None]

    @property
    def ref(self):
        """The C structure, with the parameters' present pointers."""
        for t, ptr, n in self._held:
            if t.data_ptr() != ptr or t.numel() != n:
                self._bind()
        return self._ref

    @property
    def c(self) -> ElBlockNorm:
        return self.ref._obj

    def gates(self, M: int) -> int:
        """Rows of the gate for M rows."""
        return -(-M // self.gate_rows)


def _norm_shape(norm: BlockNorm, t: torch.Tensor, name: str):
    """(shape, device) of an operand of the norm."""
    shape = M, C = tw._rows_cols(t, name)
    if C != norm.C:
        raise ValueError(f"{name} must have {norm.C} columns, got {C}")
    if M >> 31:
        tw._too_large(M, C)
    dev = _device(t, name)
    if norm.device is not None and dev != norm.device:
        raise ValueError(f"{name} must be on the parameters' device")
    return shape, dev


def _query(fn, *sizes) -> int:
    """A size query; 0 for sizes beyond the ABI's 32 bits, which it would cut."""
    return int(fn(*sizes)) if all(0 <= s < 2**31 for s in sizes) else 0


def block_norm_fwd(norm: BlockNorm, x, y=None, h=None, f: torch.Tensor = None, gate: torch.Tensor = None,
                   post_stats: torch.Tensor = None, pre_stats: torch.Tensor = None, stream=None):
    """y = x + scale gate (post_gamma post(f) + post_beta), h = pre_gamma pre(y) + pre_beta; x (or
    None: nothing added), f, y, h [M, C], gate [ceil(M / gate_rows), C] of one dtype.  Without f, h
    is the norm of x.  y or h may be None.  post_stats, pre_stats: fp32 [M, 2], written when given."""
    like = x if x is not None else f
    if like is None:
        raise ValueError("x or f must be given")
    shape, dev = _norm_shape(norm, like, "x" if x is not None else "f")
    M, C = shape
    dt = like.dtype
    xp, ldx = _mat(x, "x", shape, dt, dev)
    fp, ldf = _mat(f, "f", shape, dt, dev)
    gp, ldg = (None, C) if gate is None else _mat(gate, "gate", (norm.gates(M), C), dt, dev)
    yp, ldy = _mat(y, "y", shape, dt, dev)
    hp, ldh = _mat(h, "h", shape, dt, dev)
    _launch(lib().el_block_norm_fwd, dev, stream, norm.ref, xp, ldx, fp, ldf, gp, ldg, M, C, yp, ldy, hp, ldh,
            _vec(post_stats, "post_stats", 2 * M, dev), _vec(pre_stats, "pre_stats", 2 * M, dev), ec._dtype(like, "x"))
    return y, h


def block_norm_bwd_workspace_bytes(norm: BlockNorm, M: int) -> int:
    return _query(lib().el_block_norm_bwd_workspace_bytes, M, norm.C, norm.gate_rows)


def block_norm_bwd(norm: BlockNorm, y, dx, dy: torch.Tensor = None, dh: torch.Tensor = None, f: torch.Tensor = None,
                   gate: torch.Tensor = None, df: torch.Tensor = None, dgate: torch.Tensor = None,
                   post_stats: torch.Tensor = None, pre_stats: torch.Tensor = None, dpost_gamma: torch.Tensor = None,
                   dpost_beta: torch.Tensor = None, dpre_gamma: torch.Tensor = None, dpre_beta: torch.Tensor = None,
                   workspace: torch.Tensor = None, stream=None):
    """Gradients of block_norm_fwd from dy and / or dh, the stored y (x where f was None; may be None
    without dh), f, gate and statistics: dx, df [M, C], dgate like the gate, the parameters' fp32
    [C]; every output may be None."""
    like = dh if dh is not None else dy
    if like is None:
        raise ValueError("dy or dh must be given")
    shape, dev = _norm_shape(norm, like, "dh" if dh is not None else "dy")
    M, C = shape
    dt, gates = like.dtype, (norm.gates(M), C)
    dyp, lddy = _mat(dy, "dy", shape, dt, dev)
    dhp, lddh = _mat(dh, "dh", shape, dt, dev)
    yp, ldy = _mat(y, "y", shape, dt, dev)
    fp, ldf = _mat(f, "f", shape, dt, dev)
    gp, ldg = _mat(gate, "gate", gates, dt, dev)
    dxp, lddx = _mat(dx, "dx", shape, dt, dev)
    dfp, lddf = _mat(df, "df", shape, dt, dev)
    dgp, lddg = _mat(dgate, "dgate", gates, dt, dev)
    wsp, wsn, keep = _workspace(workspace, lambda: block_norm_bwd_workspace_bytes(norm, M), like, dev, stream)
    _launch(lib().el_block_norm_bwd, dev, stream, norm.ref, dyp, lddy, dhp, lddh, yp, ldy, fp, ldf, gp, ldg, M, C,
            _vec(post_stats, "post_stats", 2 * M, dev), _vec(pre_stats, "pre_stats", 2 * M, dev), dxp, lddx, dfp, lddf,
            dgp, lddg, _vec(dpost_gamma, "dpost_gamma", C, dev), _vec(dpost_beta, "dpost_beta", C, dev),
            _vec(dpre_gamma, "dpre_gamma", C, dev), _vec(dpre_beta, "dpre_beta", C, dev), ec._dtype(like, "dh"), wsp, wsn)
    return dx, df


class _Packed:
    """[rows, cols] values in microscaled codes: blocks of 32 columns share a scale byte."""

    def __init__(self, rows: int, cols: int, device):
        if not 0 <= rows < 2**31 or not 1 <= cols < 2**31:
            raise ValueError(f"rows must be from 0 and cols from 1 to 2^31 - 1, got {rows} x {cols}")
        self.rows, self.cols = int(rows), int(cols)
        codes, scales = self._shapes()
        self._codes = torch.empty(codes, dtype=torch.uint8, device=device)
        self._scales = torch.empty(scales, dtype=torch.uint8, device=device)
        self.device = _device(self._codes, "the packed array")

    @property
    def ptrs(self):
        return (self._codes.data_ptr(), self._scales.data_ptr()) if self.rows else (None, None)

    # (views: they share the array's memory, but giving one other storage does not take it from the array)
    @property
    def codes(self) -> torch.Tensor:
        return self._codes.detach()

    @property
    def scales(self) -> torch.Tensor:
        return self._scales.detach()

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


class Checkpoint(_Packed):
    """Activations kept in 8 bits (e4m3): codes [rows, cols rounded up to 32], scales [rows, blocks]."""

    def __init__(self, rows: int, cols: int, device="cuda"):
        super().__init__(rows, cols, device)

    def _shapes(self):
        blocks = -(-self.cols // MICRO_BLOCK)
        return (self.rows, blocks * MICRO_BLOCK), (self.rows, blocks)


class Fp4(_Packed):
    """Weights in 4 bits (e2m1), two to a byte, in the order that the matrix instructions take: tiles
    of 32 rows by 128 columns (codes) and by 512 (scales)."""

    def __init__(self, rows: int, cols: int, device="cuda"):
        super().__init__(rows, cols, device)

    def _shapes(self):
        tiles = -(-self.rows // 32)
        return (tiles, -(-self.cols // 128), 2, 64, 16), (tiles, -(-self.cols // 512), 2, 64, 4)


def _packed(p, kind, name: str, rows: int, cols: int, dev: int):
    """Pointers of a packed operand of `kind`; (None, None) of None."""
    if p is None:
        return None, None
    if type(p) is not kind:
        raise ValueError(f"{name} must be a {kind.__name__}")
    if p.rows != rows or p.cols != cols:
        raise ValueError(f"{name} must be {[rows, cols]}, got {[p.rows, p.cols]}")
    if p.device != dev:
        raise ValueError(f"{name} must be on device {dev}, got {p.codes.device}")
    return p.ptrs


def _with_packed(t: torch.Tensor, name: str, p, kind, pname: str):
    """(shape, device, pointer, row stride) of t and the pointers of a packed operand of its shape."""
    shape = M, K = tw._rows_cols(t, name)
    if (M | K) >> 31:
        tw._too_large(M, K)
    dev = _device(t, name)
    return shape, dev, _mat(t, name, shape, t.dtype, dev), _packed(p, kind, pname, M, K, dev)


def ckpt_pack(x: torch.Tensor, ckpt: Checkpoint, stream=None) -> Checkpoint:
    """Keeps x [M, K] (fp32, fp16, bf16) in 8 bits."""
    (M, K), dev, (xp, ldx), (codes, scales) = _with_packed(x, "x", ckpt, Checkpoint, "ckpt")
    _launch(lib().el_ckpt_pack, dev, stream, xp, ldx, M, K, ec._dtype(x, "x"), codes, scales)
    return ckpt


def ckpt_act_dropout_fwd(ckpt: Checkpoint, y: torch.Tensor, act: str = "none", dropout=None, stream=None):
    """y = drop(act(kept values)): what act_dropout_fwd gives on them; with neither, the kept values."""
    (M, K), dev, (yp, ldy), (codes, scales) = _with_packed(y, "y", ckpt, Checkpoint, "ckpt")
    _launch(lib().el_ckpt_act_dropout_fwd, dev, stream, codes, scales, M, K, tw._act(act), _drop(dropout, dev), yp, ldy,
            ec._dtype(y, "y"))
    return y


def ckpt_act_dropout_bwd(dy: torch.Tensor, ckpt: Checkpoint, dx: torch.Tensor, act: str = "none", dropout=None,
                         stream=None):
    """dx = drop(dy * act'(kept values)), the mask of the forward with the same dropout."""
    shape, dev, (dp, lddy), (codes, scales) = _with_packed(dy, "dy", ckpt, Checkpoint, "ckpt")
    op, lddx = _mat(dx, "dx", shape, dy.dtype, dev)
    _launch(lib().el_ckpt_act_dropout_bwd, dev, stream, dp, lddy, codes, scales, *shape, tw._act(act), _drop(dropout, dev),
            op, lddx, ec._dtype(dy, "dy"))
    return dx


def dense_bwd_ckpt_workspace_bytes(M: int, K: int, N: int) -> int:
    return _query(lib().el_dense_bwd_ckpt_workspace_bytes, M, K, N)


def dense_bwd_ckpt(x: Checkpoint, w: torch.Tensor, dz: torch.Tensor, dw: torch.Tensor, db: torch.Tensor = None,
                   dx: torch.Tensor = None, dres: torch.Tensor = None, dzb: torch.Tensor = None, pre: Checkpoint = None,
                   act: str = "none", dropout=None, workspace: torch.Tensor = None, stream=None):
    """dense_bwd with x [M, K] and pre [M, K] kept in 8 bits."""
    M, N = tw._rows_cols(dz, "dz")
    K = tw._rows_cols(w, "w")[1]
    if (M | K | N) >> 31:
        tw._too_large(M, K, N)
    dev, dt = _device(dz, "dz"), dz.dtype
    if w.shape != (N, K) or w.dtype is not dt or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"w must be contiguous [{N}, K] of {dt} on {dz.device}")
    xc, xs = _packed(x, Checkpoint, "x", M, K, dev)
    pc, ps = _packed(pre, Checkpoint, "pre", M, K, dev)
    zp, ldz = _mat(dz, "dz", (M, N), dt, dev)
    dxp, lddx = _mat(dx, "dx", (M, K), dt, dev)
    rp, ldr = _mat(dres, "dres", (M, K), dt, dev)
    bp, ldb = _mat(dzb, "dzb", (M, K), dt, dev)
    wsp, wsn, keep = _workspace(workspace, lambda: dense_bwd_ckpt_workspace_bytes(M, K, N), dz, dev, stream)
    _launch(lib().el_dense_bwd_ckpt, dev, stream, xc, xs, M, K, w.data_ptr(), N, zp, ldz, rp, ldr, dxp, lddx,
            tw._act(act), _drop(dropout, dev), pc, ps, bp, ldb, _vec(dw, "dw", N * K, dev), _vec(db, "db", N, dev),
            ec._dtype(dz, "dz"), wsp, wsn)
    return dx, dw, db


def fp4_pack(x: torch.Tensor, packed: Fp4, stream=None) -> Fp4:
    """Rounds x [M, K] (fp32, fp16, bf16) to 4 bits."""
    (M, K), dev, (xp, ldx), (codes, scales) = _with_packed(x, "x", packed, Fp4, "packed")
    _launch(lib().el_fp4_pack, dev, stream, xp, ldx, M, K, ec._dtype(x, "x"), codes, scales)
    return packed


def fp4_unpack(packed: Fp4, y: torch.Tensor, stream=None):
    """The values that the codes stand for."""
    (M, K), dev, (yp, ldy), (codes, scales) = _with_packed(y, "y", packed, Fp4, "packed")
    _launch(lib().el_fp4_unpack, dev, stream, codes, scales, M, K, yp, ldy, ec._dtype(y, "y"))
    return y


def dense_fwd_fp4_workspace_bytes(M: int, K: int, N: int) -> int:
    return _query(lib().el_dense_fwd_fp4_workspace_bytes, M, K, N)


def dense_fwd_fp4(x: torch.Tensor, w: Fp4, bias, y: torch.Tensor, act: str = "none", residual: torch.Tensor = None,
                  workspace: torch.Tensor = None, stream=None):
    """y = residual + act(x4 @ w4.T + bias), x [M, K] (bf16, fp16) rounded to 4 bits within the call,
    w a packed [N, K]; bias fp32 [N] or None; y, residual [M, N]."""
    shape = M, K = tw._rows_cols(x, "x")
    out = tw._rows_cols(y, "y")
    N = out[1]
    if (M | K | N) >> 31:
        tw._too_large(M, K, N)
    dev, dt = _device(x, "x"), x.dtype
    wc, wsc = _packed(w, Fp4, "w", N, K, dev)
    xp, ldx = _mat(x, "x", shape, dt, dev)
    rp, ldr = _mat(residual, "residual", (M, N), dt, dev)
    yp, ldy = _mat(y, "y", (M, N), dt, dev)
    wsp, wsn, keep = _workspace(workspace, lambda: dense_fwd_fp4_workspace_bytes(M, K, N), x, dev, stream)
    _launch(lib().el_dense_fwd_fp4, dev, stream, xp, ldx, M, K, wc, wsc, _vec(bias, "bias", N, dev), N, tw._act(act), rp,
            ldr, yp, ldy, ec._dtype(x, "x"), wsp, wsn)
    return y

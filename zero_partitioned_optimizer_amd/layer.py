"""The layer operators of libzero: a linear layer's products, dropout and norms.

Between the fetch of a layer's tensors (``zero_gather_tensors``) and the optimizer
step: the product with the fetched weights and its epilogue, its gradient by the
layer's input, its gradient by the weights into the flat gradient buffer whose
slices are the step's replicas, dropout with a mask that is recomputed and
never stored, and the norm of a block's rows with its gradient. The functions keep the C names of ``include/zero_layer.h`` and take torch
tensors on the current device: 2-D matrices whose rows may be longer than their
columns (``stride(0) >= size(1)``, ``stride(1) == 1``). Outputs that are not given
are allocated, and a workspace that is not given is allocated for the call, both on
the call's stream.
``FlatLinear`` puts them together for one linear layer of a flat parameter buffer,
``FlatNorm`` for one norm.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence

import torch

from . import _binding as B
from ._binding import f64, i32, i64, sz, vp

ZERO_W_OUT_IN, ZERO_W_IN_OUT = 0, 1
ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_GELU, ZERO_ACT_SILU = 0, 1, 2, 3
ZERO_LINEAR_FORWARD, ZERO_LINEAR_GRAD_INPUT, ZERO_LINEAR_GRAD_WEIGHT = 0, 1, 2
ZERO_NORM_LAYER, ZERO_NORM_RMS = 0, 1
u64 = ctypes.c_uint64

_TYPES = {torch.bfloat16: B.ZERO_BF16, torch.float32: B.ZERO_F32}


class zero_dropout(ctypes.Structure):
    """Dropout of a matrix: probability, the generator's seed and offset, and an
    optional device int64 tensor that is added to the offset when a kernel runs.
    The backward pass takes an equal one."""

    _fields_ = [("p", f64), ("seed", u64), ("offset", u64), ("counter_dev", vp)]

    def __init__(self, p: float = 0.0, seed: int = 0, offset: int = 0,
                 counter: Optional[torch.Tensor] = None):
        super().__init__(p, seed, offset, None)
        self.counter = None
        if counter is not None:
            if counter.dtype != torch.int64 or counter.numel() < 1 or not counter.is_cuda:
                raise B.ZeroError(B.ZERO_E_INVAL, "zero_dropout: counter is not an int64 device tensor")
            self.counter = counter
            self.counter_dev = counter.data_ptr()


class zero_linear_args(ctypes.Structure):
    _fields_ = [("M", i64), ("K", i64), ("N", i64), ("x", vp), ("ld_x", i64), ("w", vp),
                ("ld_w", i64), ("w_layout", i32), ("act", i32), ("bias", vp), ("residual", vp),
                ("ld_residual", i64), ("y", vp), ("ld_y", i64), ("y_dtype", i32),
                ("reserved", i32), ("preact", vp), ("ld_preact", i64), ("dropout", zero_dropout),
                ("workspace_dev", vp), ("ws_bytes", sz)]


class zero_linear_grad_input_args(ctypes.Structure):
    _fields_ = [("M", i64), ("K", i64), ("N", i64), ("dz", vp), ("ld_dz", i64), ("w", vp),
                ("ld_w", i64), ("w_layout", i32), ("act", i32), ("preact", vp), ("ld_preact", i64),
                ("dx", vp), ("ld_dx", i64), ("dx_dtype", i32), ("reserved", i32),
                ("dropout", zero_dropout), ("workspace_dev", vp), ("ws_bytes", sz)]


class zero_linear_grad_weight_args(ctypes.Structure):
    _fields_ = [("M", i64), ("K", i64), ("N", i64), ("dz", vp), ("ld_dz", i64), ("x", vp),
                ("ld_x", i64), ("dw", vp), ("ld_dw", i64), ("dbias", vp), ("w_layout", i32),
                ("grad_dtype", i32), ("accumulate", i32), ("reserved", i32),
                ("workspace_dev", vp), ("ws_bytes", sz)]


class zero_dropout_args(ctypes.Structure):
    _fields_ = [("M", i64), ("N", i64), ("x", vp), ("ld_x", i64), ("residual", vp),
                ("ld_residual", i64), ("preact", vp), ("ld_preact", i64), ("y", vp), ("ld_y", i64),
                ("x_dtype", i32), ("y_dtype", i32), ("act", i32), ("reserved", i32),
                ("dropout", zero_dropout)]


class zero_norm_args(ctypes.Structure):
    _fields_ = [("M", i64), ("N", i64), ("x", vp), ("ld_x", i64), ("residual", vp), ("ld_residual", i64),
                ("weight", vp), ("bias", vp), ("y", vp), ("ld_y", i64), ("sum", vp), ("ld_sum", i64),
                ("stats", vp), ("x_dtype", i32), ("sum_dtype", i32), ("y_dtype", i32), ("kind", i32),
                ("eps", f64)]


class zero_norm_grad_args(ctypes.Structure):
    _fields_ = [("M", i64), ("N", i64), ("dy", vp), ("ld_dy", i64), ("x", vp), ("ld_x", i64), ("weight", vp),
                ("stats", vp), ("residual_grad", vp), ("ld_residual_grad", i64), ("dx", vp), ("ld_dx", i64),
                ("dweight", vp), ("dbias", vp), ("dy_dtype", i32), ("x_dtype", i32), ("dx_dtype", i32),
                ("grad_dtype", i32), ("kind", i32), ("accumulate", i32), ("workspace_dev", vp),
                ("ws_bytes", sz)]


assert ctypes.sizeof(zero_dropout) == 32

# The argument blocks above as struct formats: the calls below fill theirs in one
# go, which a ctypes structure would do field by field.
_DROP = "dQQQ"
_FORWARD = struct.Struct("@qqqQqQqiiQQqQqiiQq" + _DROP + "QQ")
_GRAD_INPUT = struct.Struct("@qqqQqQqiiQqQqii" + _DROP + "QQ")
_GRAD_WEIGHT = struct.Struct("@qqqQqQqQqQiiiiQQ")
_DROPOUT = struct.Struct("@qqQqQqQqQqiiii" + _DROP)
_NORM = struct.Struct("@qqQqQqQQQqQqQiiiid")
_NORM_GRAD = struct.Struct("@qqQqQqQQQqQqQQiiiiiiQQ")
assert _FORWARD.size == ctypes.sizeof(zero_linear_args)
assert _GRAD_INPUT.size == ctypes.sizeof(zero_linear_grad_input_args)
assert _GRAD_WEIGHT.size == ctypes.sizeof(zero_linear_grad_weight_args)
assert _DROPOUT.size == ctypes.sizeof(zero_dropout_args)
assert _NORM.size == ctypes.sizeof(zero_norm_args)
assert _NORM_GRAD.size == ctypes.sizeof(zero_norm_grad_args)

_NO_DROP = (0.0, 0, 0, 0)
_BF16, _F32 = torch.bfloat16, torch.float32
_declared: Optional[ctypes.CDLL] = None
_call: dict = {}


def _lib() -> ctypes.CDLL:
    global _declared
    if _declared is None:
        L = B.lib()
        P = ctypes.POINTER
        for name, args in (("zero_linear_forward", zero_linear_args),
                           ("zero_linear_grad_input", zero_linear_grad_input_args),
                           ("zero_linear_grad_weight", zero_linear_grad_weight_args),
                           ("zero_dropout_add", zero_dropout_args),
                           ("zero_dropout_grad", zero_dropout_args),
                           ("zero_norm_forward", zero_norm_args),
                           ("zero_norm_grad", zero_norm_grad_args)):
            getattr(L, name).argtypes = [P(args), vp]
            getattr(L, name).restype = ctypes.c_int
            # the same entry point, for an argument block that is packed already
            _call[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, vp)((name, L))
        L.zero_linear_workspace_bytes.argtypes = [i32, i32, i64, i64, i64]
        L.zero_linear_workspace_bytes.restype = sz
        L.zero_norm_workspace_bytes.argtypes = [i64, i64]
        L.zero_norm_workspace_bytes.restype = sz
        _declared = L
    return _declared


def _enqueue(name: str, block: bytes, stream) -> None:
    if _declared is None:
        _lib()
    if stream is None:
        stream = _raw_stream()
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    rc = _call[name](block, stream)
    if rc:
        B._check(rc)


# The current device and its stream's handle, by torch's own short ways to them.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream() -> int:
    if _current is not None:
        return _current(_device())
    return torch.cuda.current_stream().cuda_stream


def _bad(fn: str, what: str):
    raise B.ZeroError(B.ZERO_E_INVAL, f"{fn}: {what}")


def _on_device(fn: str, name: str, t: torch.Tensor) -> int:
    """The device of a call's first tensor, which is the current one."""
    d = t.get_device()
    if d < 0 or d != _device():
        _bad(fn, f"{name} is on {t.device}, not on the current device")
    return d


def _mat(fn: str, name: str, t: torch.Tensor, dtype, device: int, rows: int = -1, cols: int = -1):
    """(address, ld) of a 2-D tensor after checking its type, shape, strides and device."""
    if t.dtype is not dtype:
        _bad(fn, f"{name} is {t.dtype}, not {dtype}")
    shape = t.shape
    if len(shape) != 2 or (rows >= 0 and shape[0] != rows) or (cols >= 0 and shape[1] != cols):
        _bad(fn, f"{name} has shape {tuple(shape)}, not ({rows if rows >= 0 else 'M'}, "
                 f"{cols if cols >= 0 else 'N'})")
    if t.get_device() != device:
        _bad(fn, f"{name} is on {t.device}, not on the current device")
    r, c = shape
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        _bad(fn, f"{name} has column stride {s1}; its rows must be contiguous")
    if r <= 1 or c == 0:
        return t.data_ptr(), c
    if s0 < c:
        _bad(fn, f"{name} has row stride {s0} below its {c} columns")
    return t.data_ptr(), s0


def _vec(fn: str, name: str, t: torch.Tensor, dtype, device: int, n: int) -> int:
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _bad(fn, f"{name} is {t.dtype} of shape {tuple(t.shape)}, not {n} contiguous {dtype}")
    if t.get_device() != device:
        _bad(fn, f"{name} is on {t.device}, not on the current device")
    return t.data_ptr()


def _type(fn: str, name: str, dtype) -> int:
    ty = _TYPES.get(dtype)
    if ty is None:
        _bad(fn, f"{name} is {dtype}, neither torch.bfloat16 nor torch.float32")
    return ty


def _drop(fn: str, dropout, device: int):
    if dropout is None:
        return _NO_DROP
    counter = dropout.counter_dev
    if counter and dropout.counter is not None and dropout.counter.get_device() != device:
        _bad(fn, f"the dropout's counter is on {dropout.counter.device}, not on the current device")
    return dropout.p, dropout.seed, dropout.offset, counter or 0


@functools.lru_cache(maxsize=4096)
def _workspace_need(kind: int, w_layout: int, M: int, K: int, N: int) -> int:
    return int(_lib().zero_linear_workspace_bytes(kind, w_layout, M, K, N))


def zero_linear_workspace_bytes(kind: int, w_layout: int, M: int, K: int, N: int) -> int:
    return _workspace_need(int(kind), int(w_layout), int(M), int(K), int(N))


def _new(shape, dtype, device: int, stream):
    """A new tensor from torch's allocator for use on ``stream``: memory that a call
    gives back (its workspace) goes to that stream's pool, whose order keeps later
    use behind the call's kernels."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=_cuda(device))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=_cuda(device))


def _new_like(x: torch.Tensor, dtype, device: int, stream):
    """The same in x's shape, by torch's shorter way where there is one (1.2 against 1.7 us)."""
    if stream is None and dtype is x.dtype and x.is_contiguous():
        return torch.empty_like(x)
    return _new(x.shape, dtype, device, stream)


@functools.lru_cache(maxsize=64)
def _cuda(device: int) -> torch.device:
    return torch.device("cuda", device)


def _workspace(fn: str, kind: int, w_layout: int, M: int, K: int, N: int, given, device: int, stream):
    """(address, bytes, tensor) of a product's workspace."""
    return _scratch(fn, lambda: _workspace_need(kind, w_layout, M, K, N), given, device, stream)


def _scratch(fn: str, bytes_needed, given, device: int, stream):
    """(address, bytes, tensor) of a call's workspace: the given one, or a new one."""
    if given is not None:
        if given.get_device() != device:
            _bad(fn, f"workspace is on {given.device}, not on the current device")
        if not given.is_contiguous():
            _bad(fn, "workspace is not contiguous")
        return given.data_ptr(), given.numel() * given.element_size(), given
    need = bytes_needed()
    if need == 0:
        return 0, 0, None
    ws = _new(need, torch.uint8, device, stream)
    return ws.data_ptr(), need, ws


def _weight(fn: str, name: str, w: torch.Tensor, w_layout: int, dtype, device: int, K: int, N: int):
    if w_layout == ZERO_W_OUT_IN:
        return _mat(fn, name, w, dtype, device, N, K)
    if w_layout == ZERO_W_IN_OUT:
        return _mat(fn, name, w, dtype, device, K, N)
    _bad(fn, f"unknown w_layout {w_layout}")


def zero_linear_forward(x, w, bias=None, *, w_layout: int = ZERO_W_OUT_IN, act: int = ZERO_ACT_NONE,
                        dropout: Optional[zero_dropout] = None, residual=None, y=None, preact=None,
                        dtype=None, workspace=None, stream=None):
    """y = residual + D(act(x W^T + bias)). ``preact``: a bf16 [M, N] tensor that
    receives x W^T + bias, or True for a new one, and (y, preact) is returned.
    ``dtype`` (bfloat16 or float32) is that of a new y."""
    fn = "zero_linear_forward"
    dev = _on_device(fn, "x", x)
    px, ldx = _mat(fn, "x", x, _BF16, dev)
    M, K = x.shape
    if w.dim() != 2:
        _bad(fn, f"w has shape {tuple(w.shape)}")
    N = w.shape[0] if w_layout == ZERO_W_OUT_IN else w.shape[1]
    pw, ldw = _weight(fn, "w", w, w_layout, _BF16, dev, K, N)
    if y is None:
        y = _new((M, N), dtype or (residual.dtype if residual is not None else _BF16), dev, stream)
    elif dtype is not None and y.dtype is not dtype:
        _bad(fn, f"y is {y.dtype}, not {dtype}")
    ty = _type(fn, "y", y.dtype)
    py, ldy = _mat(fn, "y", y, y.dtype, dev, M, N)
    pr = ldr = pz = ldz = pb = 0
    if residual is not None:
        pr, ldr = _mat(fn, "residual", residual, y.dtype, dev, M, N)
    both = preact is not None and preact is not False
    if both:
        if preact is True:
            preact = _new((M, N), _BF16, dev, stream)
        pz, ldz = _mat(fn, "preact", preact, _BF16, dev, M, N)
    if bias is not None:
        pb = _vec(fn, "bias", bias, _BF16, dev, N)
    ws, nws, keep = _workspace(fn, ZERO_LINEAR_FORWARD, w_layout, M, K, N, workspace, dev, stream)
    _enqueue(fn, _FORWARD.pack(M, K, N, px, ldx, pw, ldw, w_layout, act, pb, pr, ldr, py, ldy, ty, 0, pz, ldz,
                               *_drop(fn, dropout, dev), ws, nws), stream)
    return (y, preact) if both else y


def zero_linear_grad_input(dz, w, *, w_layout: int = ZERO_W_OUT_IN, act: int = ZERO_ACT_NONE, preact=None,
                           dropout: Optional[zero_dropout] = None, dx=None, dtype=None, workspace=None,
                           stream=None):
    """dx = D'(dz W) * act'(preact); ``preact`` and ``dropout`` are those of the
    layer below, whose output this layer's input was."""
    fn = "zero_linear_grad_input"
    dev = _on_device(fn, "dz", dz)
    pd, ldd = _mat(fn, "dz", dz, _BF16, dev)
    M, N = dz.shape
    if w.dim() != 2:
        _bad(fn, f"w has shape {tuple(w.shape)}")
    K = w.shape[1] if w_layout == ZERO_W_OUT_IN else w.shape[0]
    pw, ldw = _weight(fn, "w", w, w_layout, _BF16, dev, K, N)
    if dx is None:
        dx = _new((M, K), dtype or _BF16, dev, stream)
    elif dtype is not None and dx.dtype is not dtype:
        _bad(fn, f"dx is {dx.dtype}, not {dtype}")
    ty = _type(fn, "dx", dx.dtype)
    px, ldx = _mat(fn, "dx", dx, dx.dtype, dev, M, K)
    pz, ldz = _mat(fn, "preact", preact, _BF16, dev, M, K) if preact is not None else (0, 0)
    ws, nws, keep = _workspace(fn, ZERO_LINEAR_GRAD_INPUT, w_layout, M, K, N, workspace, dev, stream)
    _enqueue(fn, _GRAD_INPUT.pack(M, K, N, pd, ldd, pw, ldw, w_layout, act, pz, ldz, px, ldx, ty, 0,
                                  *_drop(fn, dropout, dev), ws, nws), stream)
    return dx


def zero_linear_grad_weight(dz, x, dw, dbias=None, *, w_layout: int = ZERO_W_OUT_IN, accumulate: bool = False,
                            workspace=None, stream=None) -> None:
    """dw [+]= dz^T x in the weight's layout, and dbias [+]= the column sums of dz;
    dw and dbias are bf16 or f32 (views of a flat gradient buffer)."""
    fn = "zero_linear_grad_weight"
    dev = _on_device(fn, "dz", dz)
    pd, ldd = _mat(fn, "dz", dz, _BF16, dev)
    M, N = dz.shape
    px, ldx = _mat(fn, "x", x, _BF16, dev, M)
    K = x.shape[1]
    ty = _type(fn, "dw", dw.dtype)
    pw, ldw = _weight(fn, "dw", dw, w_layout, dw.dtype, dev, K, N)
    pb = _vec(fn, "dbias", dbias, dw.dtype, dev, N) if dbias is not None else 0
    ws, nws, keep = _workspace(fn, ZERO_LINEAR_GRAD_WEIGHT, w_layout, M, K, N, workspace, dev, stream)
    _enqueue(fn, _GRAD_WEIGHT.pack(M, K, N, pd, ldd, px, ldx, pw, ldw, pb, w_layout, ty, 1 if accumulate else 0, 0,
                                   ws, nws), stream)


def zero_dropout_add(x, dropout: Optional[zero_dropout], *, residual=None, y=None, dtype=None, stream=None):
    """y = residual + D(x) over a matrix; y (and the residual) may be of another
    type than x."""
    fn = "zero_dropout_add"
    dev = _on_device(fn, "x", x)
    tx = _type(fn, "x", x.dtype)
    px, ldx = _mat(fn, "x", x, x.dtype, dev)
    M, N = x.shape
    if y is None:
        y = _new_like(x, dtype or (residual.dtype if residual is not None else x.dtype), dev, stream)
    elif dtype is not None and y.dtype is not dtype:
        _bad(fn, f"y is {y.dtype}, not {dtype}")
    ty = _type(fn, "y", y.dtype)
    py, ldy = _mat(fn, "y", y, y.dtype, dev, M, N)
    pr, ldr = _mat(fn, "residual", residual, y.dtype, dev, M, N) if residual is not None else (0, 0)
    _enqueue(fn, _DROPOUT.pack(M, N, px, ldx, pr, ldr, 0, 0, py, ldy, tx, ty, 0, 0, *_drop(fn, dropout, dev)),
             stream)
    return y


def zero_dropout_grad(dy, dropout: Optional[zero_dropout], *, act: int = ZERO_ACT_NONE, preact=None, dz=None,
                      dtype=None, stream=None):
    """dz = D'(dy) * act'(preact): the gradient of dropout behind an activation."""
    fn = "zero_dropout_grad"
    dev = _on_device(fn, "dy", dy)
    tx = _type(fn, "dy", dy.dtype)
    px, ldx = _mat(fn, "dy", dy, dy.dtype, dev)
    M, N = dy.shape
    if dz is None:
        dz = _new_like(dy, dtype or dy.dtype, dev, stream)
    elif dtype is not None and dz.dtype is not dtype:
        _bad(fn, f"dz is {dz.dtype}, not {dtype}")
    ty = _type(fn, "dz", dz.dtype)
    py, ldy = _mat(fn, "dz", dz, dz.dtype, dev, M, N)
    pz, ldz = _mat(fn, "preact", preact, _BF16, dev, M, N) if preact is not None else (0, 0)
    _enqueue(fn, _DROPOUT.pack(M, N, px, ldx, 0, 0, pz, ldz, py, ldy, tx, ty, act, 0, *_drop(fn, dropout, dev)),
             stream)
    return dz


@functools.lru_cache(maxsize=4096)
def _norm_need(M: int, N: int) -> int:
    return int(_lib().zero_norm_workspace_bytes(M, N))


def zero_norm_workspace_bytes(M: int, N: int) -> int:
    return _norm_need(int(M), int(N))


def zero_norm_forward(x, weight=None, bias=None, *, kind: int = ZERO_NORM_LAYER, eps: float = 1e-5, residual=None,
                      sum=None, y=None, stats=None, dtype=None, stream=None):
    """The norm of each row of x, or of s = residual + x. Returns y; with a residual or
    with stats a tuple (y, s, stats) of those that there are. ``sum``: the tensor that
    receives s (of the residual's type; new if None). ``stats``: a float32 [M, 2] tensor
    that receives each row's mean and 1 / standard deviation, which the gradient takes, or
    True for a new one. ``dtype`` is that of a new y (x's by default)."""
    fn = "zero_norm_forward"
    dev = _on_device(fn, "x", x)
    tx = _type(fn, "x", x.dtype)
    px, ldx = _mat(fn, "x", x, x.dtype, dev)
    M, N = x.shape
    if y is None:
        y = _new_like(x, dtype or x.dtype, dev, stream)
    elif dtype is not None and y.dtype is not dtype:
        _bad(fn, f"y is {y.dtype}, not {dtype}")
    ty = _type(fn, "y", y.dtype)
    py, ldy = _mat(fn, "y", y, y.dtype, dev, M, N)
    pr = ldr = ps = lds = pt = pw = pb = ts = 0
    if residual is not None:
        ts = _type(fn, "residual", residual.dtype)
        pr, ldr = _mat(fn, "residual", residual, residual.dtype, dev, M, N)
        if sum is None:
            sum = _new_like(residual, residual.dtype, dev, stream)
        ps, lds = _mat(fn, "sum", sum, residual.dtype, dev, M, N)
    elif sum is not None:
        _bad(fn, "a sum without a residual")
    if weight is not None:
        pw = _vec(fn, "weight", weight, _BF16, dev, N)
    if bias is not None:
        pb = _vec(fn, "bias", bias, _BF16, dev, N)
    if stats is False:
        stats = None
    if stats is not None:
        if stats is True:
            stats = _new((M, 2), _F32, dev, stream)
        pt = _stats(fn, stats, dev, M)
    _enqueue(fn, _NORM.pack(M, N, px, ldx, pr, ldr, pw, pb, py, ldy, ps, lds, pt, tx, ts, ty, kind, eps), stream)
    if residual is None:
        return y if stats is None else (y, stats)
    return (y, sum) if stats is None else (y, sum, stats)


def _stats(fn: str, t: torch.Tensor, device: int, M: int) -> int:
    if M == 0 and t.numel() == 0:       # whatever its strides say
        return 0
    p, ld = _mat(fn, "stats", t, _F32, device, M, 2)
    if ld != 2:
        _bad(fn, f"stats has row stride {ld}, not 2")
    return p


def zero_norm_grad(dy, x, weight=None, stats=None, *, kind: int = ZERO_NORM_LAYER, residual_grad=None, dx=None,
                   dtype=None, dweight=None, dbias=None, accumulate: bool = False, workspace=None, stream=None):
    """dx = residual_grad + the norm's gradient by its rows, from dy, the rows x that were
    normed (s, where there was a residual) and their stats; and, where they are given,
    dweight and dbias [+]= the gradients by weight and bias (bf16 or f32, views of a flat
    gradient buffer). ``dtype`` is that of a new dx (the residual_grad's, or dy's, by default)."""
    fn = "zero_norm_grad"
    dev = _on_device(fn, "dy", dy)
    td = _type(fn, "dy", dy.dtype)
    pd, ldd = _mat(fn, "dy", dy, dy.dtype, dev)
    M, N = dy.shape
    tx = _type(fn, "x", x.dtype)
    px, ldx = _mat(fn, "x", x, x.dtype, dev, M, N)
    if stats is None:
        _bad(fn, "stats of the forward pass are missing")
    pt = _stats(fn, stats, dev, M)
    if dx is None:
        dx = _new_like(dy, dtype or (residual_grad.dtype if residual_grad is not None else dy.dtype), dev, stream)
    elif dtype is not None and dx.dtype is not dtype:
        _bad(fn, f"dx is {dx.dtype}, not {dtype}")
    to = _type(fn, "dx", dx.dtype)
    po, ldo = _mat(fn, "dx", dx, dx.dtype, dev, M, N)
    pr = ldr = pw = pgw = pgb = ws = nws = tg = 0
    if residual_grad is not None:
        pr, ldr = _mat(fn, "residual_grad", residual_grad, dx.dtype, dev, M, N)
    if weight is not None:
        pw = _vec(fn, "weight", weight, _BF16, dev, N)
    if dweight is not None:
        tg = _type(fn, "dweight", dweight.dtype)
        pgw = _vec(fn, "dweight", dweight, dweight.dtype, dev, N)
    if dbias is not None:
        tg = _type(fn, "dbias", dbias.dtype)
        pgb = _vec(fn, "dbias", dbias, dbias.dtype if dweight is None else dweight.dtype, dev, N)
    if dweight is not None or dbias is not None:
        ws, nws, keep = _scratch(fn, lambda: _norm_need(M, N), workspace, dev, stream)
    _enqueue(fn, _NORM_GRAD.pack(M, N, pd, ldd, px, ldx, pw, pt, pr, ldr, po, ldo, pgw, pgb, td, tx, to, tg, kind,
                                 1 if accumulate else 0, ws, nws), stream)
    return dx


class FlatLinear:
    """One linear layer of a model whose parameters and gradients lie in flat
    buffers: tensors ``weight`` and ``bias`` (indices, bias optional) of a layout,
    ``inputs`` by ``outputs``.

    ``fetch`` copies the layer's tensors out of the rank shards (stage 3); or
    ``use`` takes them from a whole bf16 parameter buffer. ``forward`` and
    ``backward`` then run the layer, and ``backward`` writes or accumulates the
    weight and bias gradients in place at the tensors' offsets of a flat gradient
    buffer, whose slice [r S, (r + 1) S) is this rank's gradient replica for the
    step of rank r."""

    def __init__(self, offsets: Sequence[int], numels: Sequence[int], weight: int, bias: Optional[int],
                 inputs: int, outputs: int, *, w_layout: int = ZERO_W_OUT_IN, act: int = ZERO_ACT_NONE):
        if w_layout not in (ZERO_W_OUT_IN, ZERO_W_IN_OUT):
            _bad("FlatLinear", f"unknown w_layout {w_layout}")
        if numels[weight] != inputs * outputs:
            _bad("FlatLinear", f"tensor {weight} holds {numels[weight]} elements, not {inputs} x {outputs}")
        if bias is not None and numels[bias] != outputs:
            _bad("FlatLinear", f"tensor {bias} holds {numels[bias]} elements, not {outputs}")
        self.K, self.N, self.w_layout, self.act = int(inputs), int(outputs), int(w_layout), int(act)
        self.w_off = int(offsets[weight])
        self.b_off = None if bias is None else int(offsets[bias])
        self._shape = (self.N, self.K) if w_layout == ZERO_W_OUT_IN else (self.K, self.N)
        self.w = self.b = None

    def _views(self, flat: torch.Tensor):
        n = self.K * self.N
        if flat.dim() != 1 or flat.stride(0) != 1 or flat.numel() < self.w_off + n or (
                self.b_off is not None and flat.numel() < self.b_off + self.N):
            _bad("FlatLinear", f"a flat buffer of shape {tuple(flat.shape)} does not hold the layer's tensors")
        w = flat[self.w_off:self.w_off + n].view(self._shape)
        return w, None if self.b_off is None else flat[self.b_off:self.b_off + self.N]

    def use(self, params: torch.Tensor) -> None:
        """Take the layer's tensors from a flat bf16 parameter buffer (no copy)."""
        self.w, self.b = self._views(params)

    def fetch(self, shards, shard_S: int, stream=None) -> None:
        """Copy the layer's tensors out of the rank shards (bf16 or its bit patterns). Passes
        may run on the copies' stream, or on the current one once it waits for that."""
        offs = [self.w_off] + ([] if self.b_off is None else [self.b_off])
        nums = [self.K * self.N] + ([] if self.b_off is None else [self.N])
        got = B.zero_gather_tensors(shards, shard_S, offs, nums, stream=stream)
        self.w = got[0].view(torch.bfloat16).view(self._shape)
        self.b = got[1].view(torch.bfloat16) if self.b_off is not None else None

    def release(self) -> None:
        """Drop the layer's tensors (after its pass, under stage 3)."""
        self.w = self.b = None

    def forward(self, x, *, dropout=None, residual=None, keep_preact: Optional[bool] = None, dtype=None,
                workspace=None, stream=None):
        """(y, preact): preact is None unless the activation's gradient needs it."""
        if self.w is None:
            _bad("FlatLinear.forward", "the layer's tensors are not here: fetch or use first")
        keep = self.act != ZERO_ACT_NONE if keep_preact is None else keep_preact
        got = zero_linear_forward(x, self.w, self.b, w_layout=self.w_layout, act=self.act, dropout=dropout,
                                  residual=residual, preact=keep, dtype=dtype, workspace=workspace,
                                  stream=stream)
        return got if keep else (got, None)

    def backward(self, dz, x, grads: Optional[torch.Tensor], *, accumulate: bool = False, below=None,
                 input_grad: bool = True, dtype=None, workspace=None, stream=None):
        """Gradients of the layer from dz = d loss / d (x W^T + b): the weight's and
        the bias's into ``grads`` (skipped if None), and the input's returned
        (None without ``input_grad``). ``below``: (act, preact, dropout) of the
        layer that made x, whose gradient is then taken on to its pre-activation."""
        if grads is not None:
            dw, db = self._views(grads)
            zero_linear_grad_weight(dz, x, dw, db, w_layout=self.w_layout, accumulate=accumulate,
                                    workspace=workspace, stream=stream)
        if not input_grad:
            return None
        if self.w is None:
            _bad("FlatLinear.backward", "the layer's tensors are not here: fetch or use first")
        act, preact, dropout = below if below is not None else (ZERO_ACT_NONE, None, None)
        return zero_linear_grad_input(dz, self.w, w_layout=self.w_layout, act=act, preact=preact,
                                      dropout=dropout, dtype=dtype, workspace=workspace, stream=stream)


class FlatNorm:
    """One norm of a model whose parameters and gradients lie in flat buffers: tensors
    ``weight`` and ``bias`` (indices, bias optional) of a layout, ``width`` elements each.
    ``fetch``, ``use`` and ``release`` as of ``FlatLinear``; ``backward`` writes or
    accumulates the gradients of weight and bias in place at the tensors' offsets of a
    flat gradient buffer."""

    def __init__(self, offsets: Sequence[int], numels: Sequence[int], weight: int, bias: Optional[int], width: int, *,
                 kind: int = ZERO_NORM_LAYER, eps: float = 1e-5):
        for i in (weight, bias):
            if i is not None and numels[i] != width:
                _bad("FlatNorm", f"tensor {i} holds {numels[i]} elements, not {width}")
        if kind not in (ZERO_NORM_LAYER, ZERO_NORM_RMS):
            _bad("FlatNorm", f"unknown kind {kind}")
        self.N, self.kind, self.eps = int(width), int(kind), float(eps)
        self.w_off = int(offsets[weight])
        self.b_off = None if bias is None else int(offsets[bias])
        self.w = self.b = None

    def _views(self, flat: torch.Tensor):
        offs = [self.w_off] + ([] if self.b_off is None else [self.b_off])
        if flat.dim() != 1 or flat.stride(0) != 1 or flat.numel() < max(offs) + self.N:
            _bad("FlatNorm", f"a flat buffer of shape {tuple(flat.shape)} does not hold the norm's tensors")
        got = [flat[o:o + self.N] for o in offs]
        return got[0], got[1] if self.b_off is not None else None

    def use(self, params: torch.Tensor) -> None:
        """Take the norm's tensors from a flat bf16 parameter buffer (no copy)."""
        self.w, self.b = self._views(params)

    def fetch(self, shards, shard_S: int, stream=None) -> None:
        """Copy the norm's tensors out of the rank shards (bf16 or its bit patterns). Passes
        may run on the copies' stream, or on the current one once it waits for that."""
        offs = [self.w_off] + ([] if self.b_off is None else [self.b_off])
        got = B.zero_gather_tensors(shards, shard_S, offs, [self.N] * len(offs), stream=stream)
        self.w = got[0].view(torch.bfloat16)
        self.b = got[1].view(torch.bfloat16) if self.b_off is not None else None

    def release(self) -> None:
        """Drop the norm's tensors (after its pass, under stage 3)."""
        self.w = self.b = None

    def _here(self, fn: str):
        if self.w is None:
            _bad(fn, "the norm's tensors are not here: fetch or use first")

    def forward(self, x, *, residual=None, sum=None, dtype=None, stream=None):
        """(y, s, stats): the norm of s = residual + x (x itself without a residual), and what
        ``backward`` takes."""
        self._here("FlatNorm.forward")
        got = zero_norm_forward(x, self.w, self.b, kind=self.kind, eps=self.eps, residual=residual, sum=sum,
                                stats=True, dtype=dtype, stream=stream)
        return got if residual is not None else (got[0], x, got[1])

    def backward(self, dy, s, stats, grads: Optional[torch.Tensor], *, accumulate: bool = False, residual_grad=None,
                 dx=None, dtype=None, workspace=None, stream=None):
        """The gradient by s, the residual stream's own added; the weight's and the bias's go
        into ``grads`` (skipped if None)."""
        self._here("FlatNorm.backward")
        dw, db = self._views(grads) if grads is not None else (None, None)
        return zero_norm_grad(dy, s, self.w, stats, kind=self.kind, residual_grad=residual_grad, dx=dx, dtype=dtype,
                              dweight=dw, dbias=db, accumulate=accumulate, workspace=workspace, stream=stream)

"""The step of a layer's matrices by an orthogonalised momentum, operator by operator.

Beside the Adam step, for the tensors that are matrices: the momentum of a shard, the
orthogonalisation of whole matrices by Newton-Schulz products on the matrix cores, and
the update of the shard's master copy and bf16 slot. The functions keep the C names of
``include/zero_muon.h`` and take torch tensors on the current device; outputs that are
not given are allocated, and a workspace that is not given is allocated for the call,
both on the call's stream. ``MuonShardStep`` puts them together.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence

import torch

from . import _binding as B
from ._binding import f64, i32, i64, sz, vp
from .layer import _bad, _mat, _new, _on_device, _raw_stream, _scratch, _type

ZERO_MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


class zero_muon_momentum_args(ctypes.Structure):
    _fields_ = [("n", i64), ("grad", vp), ("momentum", vp), ("u", vp), ("grad_dtype", i32), ("u_dtype", i32),
                ("nesterov", i32), ("reserved", i32), ("mu", f64), ("stats_dev", vp)]


class zero_muon_update_args(ctypes.Structure):
    _fields_ = [("n", i64), ("p", vp), ("o", vp), ("slot_bf16", vp), ("lr", f64), ("weight_decay", f64),
                ("stats_dev", vp)]


class zero_orthogonalize_args(ctypes.Structure):
    _fields_ = [("batch", i64), ("rows", i64), ("cols", i64), ("x", vp), ("ld_x", i64), ("stride_x", i64),
                ("o", vp), ("ld_o", i64), ("stride_o", i64), ("x_dtype", i32), ("steps", i32),
                ("coefficients", ctypes.POINTER(f64)), ("eps", f64), ("scale", f64), ("workspace_dev", vp),
                ("ws_bytes", sz)]


# The argument blocks as struct formats, packed in one go.
_MOMENTUM = struct.Struct("@qQQQiiiidQ")
_UPDATE = struct.Struct("@qQQQddQ")
_ORTH = struct.Struct("@qqqQqqQqqiiQddQQ")
assert _MOMENTUM.size == ctypes.sizeof(zero_muon_momentum_args)
assert _UPDATE.size == ctypes.sizeof(zero_muon_update_args)
assert _ORTH.size == ctypes.sizeof(zero_orthogonalize_args)

_BF16, _F32 = torch.bfloat16, torch.float32
_declared: Optional[ctypes.CDLL] = None
_call: dict = {}


def _lib() -> ctypes.CDLL:
    global _declared
    if _declared is None:
        L = B.lib()
        for name, args in (("zero_muon_momentum", zero_muon_momentum_args),
                           ("zero_muon_update", zero_muon_update_args),
                           ("zero_orthogonalize", zero_orthogonalize_args)):
            getattr(L, name).argtypes = [ctypes.POINTER(args), vp]
            getattr(L, name).restype = ctypes.c_int
            # the same entry point, for an argument block that is packed already
            _call[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, vp)((name, L))
        L.zero_orthogonalize_workspace_bytes.argtypes = [i64, i64, i64]
        L.zero_orthogonalize_workspace_bytes.restype = sz
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


def _flat(fn: str, name: str, t: torch.Tensor, dtypes, device: int, n: int) -> int:
    if t.dtype not in dtypes or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _bad(fn, f"{name} is {t.dtype} of shape {tuple(t.shape)}, not {n} contiguous elements of "
                 + " or ".join(str(d) for d in dtypes))
    if t.get_device() != device:
        _bad(fn, f"{name} is on {t.device}, not on the current device")
    return t.data_ptr()


def _stats(fn: str, t, device: int) -> int:
    """The address of a device zero_stats (16 bytes)."""
    if t is None:
        return 0
    if t.get_device() != device or not t.is_contiguous() or t.numel() * t.element_size() < 16:
        _bad(fn, "stats is not 16 contiguous bytes on the current device")
    return t.data_ptr()


def zero_muon_momentum(grad, momentum, *, mu: float = 0.95, nesterov: bool = True, u=None, dtype=None, stats=None,
                       stream=None):
    """momentum = mu momentum + grad in place, over flat tensors, and u = grad + mu momentum
    (or the momentum itself without ``nesterov``), returned. ``dtype`` (bfloat16 or float32)
    is that of a new u. ``stats``: a device zero_stats whose overflow flag leaves both as
    they were."""
    fn = "zero_muon_momentum"
    dev = _on_device(fn, "grad", grad)
    tg = _type(fn, "grad", grad.dtype)
    n = grad.numel()
    pg = _flat(fn, "grad", grad, (grad.dtype,), dev, n)
    pm = _flat(fn, "momentum", momentum, (_F32,), dev, n)
    if u is None:
        u = _new((n,), dtype or _BF16, dev, stream)
    elif dtype is not None and u.dtype is not dtype:
        _bad(fn, f"u is {u.dtype}, not {dtype}")
    tu = _type(fn, "u", u.dtype)
    pu = _flat(fn, "u", u, (u.dtype,), dev, n)
    _enqueue(fn, _MOMENTUM.pack(n, pg, pm, pu, tg, tu, 1 if nesterov else 0, 0, mu, _stats(fn, stats, dev)), stream)
    return u


def zero_muon_update(p, o, *, lr: float, weight_decay: float = 0.0, slot=None, stats=None, stream=None) -> None:
    """p = p (1 - lr weight_decay) - lr o in place, over flat tensors (p float32, o bfloat16),
    and slot (bfloat16, or int16 for its bit patterns) = p rounded. ``stats`` as above."""
    fn = "zero_muon_update"
    dev = _on_device(fn, "p", p)
    n = p.numel()
    pp = _flat(fn, "p", p, (_F32,), dev, n)
    po = _flat(fn, "o", o, (_BF16,), dev, n)
    ps = _flat(fn, "slot", slot, (_BF16, torch.int16), dev, n) if slot is not None else 0
    _enqueue(fn, _UPDATE.pack(n, pp, po, ps, lr, weight_decay, _stats(fn, stats, dev)), stream)


@functools.lru_cache(maxsize=4096)
def _orth_need(batch: int, rows: int, cols: int) -> int:
    return int(_lib().zero_orthogonalize_workspace_bytes(batch, rows, cols))


def zero_orthogonalize_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return _orth_need(int(batch), int(rows), int(cols))


@functools.lru_cache(maxsize=64)
def _table(coefficients, steps: int):
    """The host table of a call's coefficients: one triple for every step, or one each."""
    if coefficients is None:
        return None
    triples = coefficients if any(isinstance(t, tuple) for t in coefficients) else (coefficients,) * steps
    if len(triples) != steps or any(not isinstance(t, tuple) or len(t) != 3 for t in triples):
        _bad("zero_orthogonalize", f"coefficients are neither three numbers nor {steps} triples")
    return (f64 * (3 * steps))(*[float(v) for t in triples for v in t])


def _coefficients(c):
    """As a key of _table."""
    return None if c is None else tuple(tuple(t) if hasattr(t, "__len__") else t for t in c)


def _check_step(shapes, *, mu, nesterov, lr, weight_decay, steps, coefficients, eps) -> None:
    """Raises what the operators of a step would for these values and (rows, cols, scale) of
    its matrices: the calls themselves, with nothing to do."""
    bf16, f32 = B.ZERO_BF16, B.ZERO_F32
    _enqueue("zero_muon_momentum", _MOMENTUM.pack(0, 0, 0, 0, f32, bf16, 1 if nesterov else 0, 0, mu, 0), 0)
    _enqueue("zero_muon_update", _UPDATE.pack(0, 0, 0, 0, lr, weight_decay, 0), 0)
    table = _table(_coefficients(coefficients), int(steps)) if 1 <= steps <= 64 else None
    for rows, cols, scale in shapes:
        _enqueue("zero_orthogonalize",
                 _ORTH.pack(0, rows, cols, 0, cols, 0, 0, cols, 0, bf16, steps,
                            ctypes.addressof(table) if table is not None else 0, eps, scale, 0, 0), 0)


def _stack(fn: str, name: str, t: torch.Tensor, dtype, device: int):
    """(address, ld, batch stride) of a matrix or a stack of matrices."""
    if t.dim() == 2:
        return _mat(fn, name, t, dtype, device) + (0,)
    if t.dim() != 3:
        _bad(fn, f"{name} has shape {tuple(t.shape)}, neither a matrix nor a stack of them")
    if t.shape[0] == 0:
        return 0, t.shape[2], 0
    p, ld = _mat(fn, name, t[0], dtype, device)
    return p, ld, t.stride(0)


def zero_orthogonalize(x, *, out=None, steps: int = 5, coefficients=ZERO_MUON_COEFFICIENTS, eps: float = 1e-7,
                       scale: float = 1.0, workspace=None, stream=None):
    """scale times the nearly semi-orthogonal matrix of x [R, C], or of each matrix of a
    stack [B, R, C] (bfloat16 or float32; a row contiguous, rows at least C elements apart, and
    matrices at least as far as one reaches, so that none lies within another): X = x / (|x| +
    eps), then ``steps`` times X = a X + (b A + c A A) X with A = X X^T. ``coefficients``:
    (a, b, c), or one such triple for each step; the steps' |a|, where above 1, may multiply to
    8192 (seven steps of the default ones). Returns ``out`` (bfloat16, x's shape; new
    if None)."""
    fn = "zero_orthogonalize"
    dev = _on_device(fn, "x", x)
    tx = _type(fn, "x", x.dtype)
    px, ldx, sx = _stack(fn, "x", x, x.dtype, dev)
    if out is None:
        out = _new(x.shape, _BF16, dev, stream)
    elif out.shape != x.shape:
        _bad(fn, f"out has shape {tuple(out.shape)}, not {tuple(x.shape)}")
    po, ldo, so = _stack(fn, "out", out, _BF16, dev)
    batch, (rows, cols) = (x.shape[0] if x.dim() == 3 else 1), x.shape[-2:]
    table = _table(_coefficients(coefficients), int(steps)) if 1 <= steps <= 64 else None
    ws, nws, keep = _scratch(fn, lambda: _orth_need(batch, rows, cols), workspace, dev, stream)
    _enqueue(fn, _ORTH.pack(batch, rows, cols, px, ldx, sx, po, ldo, so, tx, steps,
                            ctypes.addressof(table) if table is not None else 0, eps, scale, ws, nws), stream)
    return out

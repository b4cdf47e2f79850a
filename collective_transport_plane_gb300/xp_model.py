"""ctypes binding of the operators of a layer in 8 bits of libxp.so (include/xp_model.h): same names, argument marshalling only.

Tensors are torch tensors (or objects with the same `data_ptr()`, `get_device()`, `shape`, `stride()` and `dtype`): their
pointers, sizes, strides and types are read off.  Shapes and types that do not belong together, and tensors that are not
on the current device, raise ValueError before the call.  Codes are torch.uint8 or torch.float8_e4m3fn, scales torch.uint8
or torch.float8_e8m0fnu.  Streams, and the errors of the library itself (`XpError`), are as in `xp`.
"""
from __future__ import annotations

import ctypes
import sys

from . import xp
from .xp import XP_BF16, XP_F32, XP_OK, XP_U8, XpError, _stream  # noqa: F401

XP_BLOCK8 = 128
XP_MODEL_MAX_ROWS = 1 << 28
XP_MODEL_MAX_COLS = 1 << 20
XP_MODEL_MAX_STRIDE = 1 << 36
XP_DISTILL_MAX_TOP = 1024

# every entry point include/xp_model.h declares
EXPORTS = [
    "xp_block8_encode", "xp_block8_decode", "xp_matmul8", "xp_matmul8_status", "xp_rmsnorm_forward", "xp_rmsnorm_workspace",
    "xp_rmsnorm_backward", "xp_distill_forward", "xp_distill_backward",
]

_lib = xp._lib
_P, _I, _Z, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
for _name, _args in {
    "xp_block8_encode": [_P, _Z, _Z, _Z, _I, _I, _P, _Z, _P, _Z, _P, _Z, _P, _Z, _P],
    "xp_block8_decode": [_P, _Z, _P, _Z, _Z, _Z, _I, _P, _Z, _I, _P],
    "xp_matmul8": [_P, _Z, _P, _Z, _I, _P, _Z, _P, _Z, _I, _P, _Z, _Z, _Z, _Z, _I, _I, _P],
    "xp_matmul8_status": [],
    "xp_rmsnorm_forward": [_P, _Z, _P, _Z, _P, _P, _Z, _P, _Z, _P, _Z, _P, _Z, _P, _Z, _Z, _F, _I, _I, _P],
    "xp_rmsnorm_workspace": [_Z, _Z, ctypes.POINTER(_Z)],
    "xp_rmsnorm_backward": [_P, _Z, _P, _Z, _P, _P, _P, _Z, _P, _Z, _P, _Z, _Z, _I, _I, _I, _P, _Z, _P],
    "xp_distill_forward": [_P, _Z, _P, _P, _Z, _Z, _Z, _F, _P, _P, _I, _P],
    "xp_distill_backward": [_P, _Z, _P, _P, _P, _P, _Z, _Z, _Z, _F, _P, _Z, _I, _P],
}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = ctypes.c_int

_FLOATS = {"torch.float32": XP_F32, "torch.bfloat16": XP_BF16}
_BYTES = ("torch.uint8", "torch.float8_e4m3fn", "torch.float8_e8m0fnu")
_types = {}   # torch dtype -> xp_dtype (XP_U8: codes and scales), filled as types are met


def _dtype(t) -> int:
    found = _types.get(t.dtype)
    if found is None:
        name = str(t.dtype)
        if name not in _FLOATS and name not in _BYTES:
            raise ValueError(f"no xp_dtype for {t.dtype}")
        found = _types[t.dtype] = _FLOATS.get(name, XP_U8)
    return found


def _current_device() -> int:
    torch = sys.modules.get("torch")
    return torch.cuda.current_device() if torch is not None else 0


def _on_device(*tensors):
    """Refuses tensors that are not on the current device."""
    at = {t.get_device() for t in tensors if t is not None}
    if len(at) > 1 or at and (min(at) < 0 or at != {_current_device()}):
        raise ValueError(f"tensors on devices {sorted(at)}, not all on the current one (-1: the host)")


def _matrix(t, rows, cols, what, dtype):
    """(address, stride) of a rows x cols matrix whose columns are side by side (None: none)."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols) or (_types.get(t.dtype) or _dtype(t)) != dtype:
        raise ValueError(f"{what} is {tuple(t.shape)} of {t.dtype}, not ({rows}, {cols}) of its type")
    stride, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}'s columns are {step} elements apart")
    return t.data_ptr(), stride


def _vector(t, n, what, dtype):
    """The address of n contiguous elements (None: none)."""
    if t is None:
        return None
    if t.numel() != n or not t.is_contiguous() or _dtype(t) != dtype:
        raise ValueError(f"{what} is not {n} contiguous elements of its type")
    return t.data_ptr()


def _block8(codes, scales, rows, cols, block_rows, what):
    """(codes, stride, scales, stride) of a matrix in 8 bits; both or neither."""
    if (codes is None) != (scales is None):
        raise ValueError(f"{what} without its scales, or scales without codes")
    if block_rows not in (1, XP_BLOCK8):
        raise ValueError(f"{what}: blocks of {block_rows} rows, neither 1 nor 128")
    return (*_matrix(codes, rows, cols, what, XP_U8),
            *_matrix(scales, -(-rows // block_rows), -(-cols // XP_BLOCK8), f"{what}'s scales", XP_U8))


def _float(t, what):
    dt = _dtype(t)
    if dt == XP_U8:
        raise ValueError(f"{what} is {t.dtype}")
    return dt


def _check(st: int, where: str):
    if st != XP_OK:
        xp._check(st, where)


def xp_block8_encode(x, codes=None, scales=None, codes_t=None, scales_t=None, block_rows: int = 1, stream=None) -> None:
    """x (rows x cols) in 8 bits into codes and scales, and its transpose into codes_t and scales_t; either pair may be None."""
    rows, cols = x.shape
    dt = _float(x, "x")
    _on_device(x, codes, scales, codes_t, scales_t)
    _check(_lib.xp_block8_encode(*_matrix(x, rows, cols, "x", dt), rows, cols, dt, block_rows, *_block8(codes, scales, rows, cols, block_rows, "codes"),
                                 *_block8(codes_t, scales_t, cols, rows, block_rows, "codes_t"), _stream(stream)), "xp_block8_encode")


def xp_block8_decode(codes, scales, out, block_rows: int = 1, stream=None) -> None:
    """The values that a matrix in 8 bits stands for, into out."""
    rows, cols = out.shape
    dt = _float(out, "out")
    _on_device(codes, scales, out)
    _check(_lib.xp_block8_decode(*_block8(codes, scales, rows, cols, block_rows, "codes"), rows, cols, block_rows, *_matrix(out, rows, cols, "out", dt), dt,
                                 _stream(stream)), "xp_block8_decode")


def xp_matmul8(a, a_scales, b, b_scales, c, a_block_rows: int = 1, b_block_rows: int = 1, accumulate: bool = False, stream=None) -> None:
    """c = a b^T (accumulate: c + a b^T) of a (m x k) and b (n x k) in 8 bits."""
    (m, k), n, dt = a.shape, b.shape[0], _float(c, "c")
    _on_device(a, a_scales, b, b_scales, c)
    pa, sa, psa, ssa = _block8(a, a_scales, m, k, a_block_rows, "a")
    pb, sb, psb, ssb = _block8(b, b_scales, n, k, b_block_rows, "b")
    _check(_lib.xp_matmul8(pa, sa, psa, ssa, a_block_rows, pb, sb, psb, ssb, b_block_rows, *_matrix(c, m, n, "c", dt), m, n, k, dt,
                           1 if accumulate else 0, _stream(stream)), "xp_matmul8")


def xp_matmul8_status() -> int:
    """Waits for the device; XP_ERR_TIMEOUT if a product ever gave up a wait, else XP_OK."""
    st = _lib.xp_matmul8_status()
    if st not in (XP_OK, xp.XP_ERR_TIMEOUT):
        xp._check(st, "xp_matmul8_status")
    return st


def xp_rmsnorm_forward(x, gamma, y=None, residual=None, added=None, rstd=None, y8=None, y8_scales=None, eps: float = 1e-5, stream=None) -> None:
    """The root-mean-square norm of x, or of x + residual (stored in added), into y, and in 8 bits into y8."""
    rows, cols = x.shape
    dt = _float(x, "x")
    wdt = dt if gamma is None else _float(gamma, "gamma")
    _on_device(x, gamma, y, residual, added, rstd, y8, y8_scales)
    _check(_lib.xp_rmsnorm_forward(*_matrix(x, rows, cols, "x", dt), *_matrix(residual, rows, cols, "residual", dt), _vector(gamma, cols, "gamma", wdt),
                                   *_matrix(added, rows, cols, "added", dt), *_matrix(y, rows, cols, "y", dt),
                                   *_block8(y8, y8_scales, rows, cols, 1, "y8"), _vector(rstd, rows, "rstd", XP_F32), rows, cols, eps, dt, wdt,
                                   _stream(stream)), "xp_rmsnorm_forward")


def xp_rmsnorm_workspace(rows: int, cols: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.xp_rmsnorm_workspace(rows, cols, ctypes.byref(out)), "xp_rmsnorm_workspace")
    return out.value


def xp_rmsnorm_backward(dy, h, gamma, rstd, dx, dgamma=None, workspace=None, dadded=None, accumulate: bool = False, stream=None) -> None:
    """dx (+ dadded), and over the rows dgamma, from dy, the norm's input h and the forward pass's rstd."""
    rows, cols = h.shape
    dt = _float(h, "h")
    wdt = dt if gamma is None else _float(gamma, "gamma")
    _on_device(dy, h, gamma, rstd, dx, dgamma, workspace, dadded)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace is not contiguous")
    work, nbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _check(_lib.xp_rmsnorm_backward(*_matrix(dy, rows, cols, "dy", dt), *_matrix(h, rows, cols, "h", dt), _vector(gamma, cols, "gamma", wdt),
                                    _vector(rstd, rows, "rstd", XP_F32), *_matrix(dadded, rows, cols, "dadded", dt),
                                    *_matrix(dx, rows, cols, "dx", dt), _vector(dgamma, cols, "dgamma", XP_F32), rows, cols, dt, wdt,
                                    1 if accumulate else 0, work, nbytes, _stream(stream)), "xp_rmsnorm_backward")


def _top(ids, teacher, rows):
    """(ids, teacher, entries per row), both rows x top side by side."""
    top = ids.shape[1]
    if ids.shape != (rows, top) or str(ids.dtype) != "torch.int32" or not ids.is_contiguous():
        raise ValueError(f"ids is {tuple(ids.shape)} of {ids.dtype}, not {rows} contiguous rows of torch.int32")
    if teacher.shape != (rows, top):
        raise ValueError(f"teacher is {tuple(teacher.shape)}, not {(rows, top)}")
    return ids.data_ptr(), _vector(teacher, rows * top, "teacher", XP_F32), top


def xp_distill_forward(logits, ids, teacher, loss, lse=None, temperature: float = 1.0, stream=None) -> None:
    """Each row's loss against the teacher's logits (rows x top, fp32) at ids (int32), and the row's log-sum-exp."""
    rows, vocab = logits.shape
    dt = _float(logits, "logits")
    _on_device(logits, ids, teacher, loss, lse)
    pi, pt, top = _top(ids, teacher, rows)
    _check(_lib.xp_distill_forward(*_matrix(logits, rows, vocab, "logits", dt), pi, pt, rows, vocab, top, temperature,
                                   _vector(loss, rows, "loss", XP_F32), _vector(lse, rows, "lse", XP_F32), dt, _stream(stream)), "xp_distill_forward")


def xp_distill_backward(logits, ids, teacher, lse, dloss, dlogits, temperature: float = 1.0, stream=None) -> None:
    """dlogits from dloss (one per row) and the forward pass's lse; dlogits may be logits."""
    rows, vocab = logits.shape
    dt = _float(logits, "logits")
    _on_device(logits, ids, teacher, lse, dloss, dlogits)
    pi, pt, top = _top(ids, teacher, rows)
    _check(_lib.xp_distill_backward(*_matrix(logits, rows, vocab, "logits", dt), pi, pt, _vector(lse, rows, "lse", XP_F32),
                                    _vector(dloss, rows, "dloss", XP_F32), rows, vocab, top, temperature,
                                    *_matrix(dlogits, rows, vocab, "dlogits", dt), dt, _stream(stream)), "xp_distill_backward")

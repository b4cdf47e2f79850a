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

_encode, _decode, _matmul, _forward, _backward, _distill, _distill_back = (
    _lib.xp_block8_encode, _lib.xp_block8_decode, _lib.xp_matmul8, _lib.xp_rmsnorm_forward, _lib.xp_rmsnorm_backward, _lib.xp_distill_forward,
    _lib.xp_distill_backward)

_FLOATS = {"torch.float32": XP_F32, "torch.bfloat16": XP_BF16}
_BYTES = ("torch.uint8", "torch.float8_e4m3fn", "torch.float8_e8m0fnu")


class _Types(dict):
    """torch dtype -> xp_dtype (XP_U8: codes and scales), filled as types are met."""

    def __missing__(self, dtype):
        name = str(dtype)
        if name not in _FLOATS and name not in _BYTES:
            raise ValueError(f"no xp_dtype for {dtype}")
        found = self[dtype] = _FLOATS.get(name, XP_U8)
        return found


class _Bytes(dict):
    """torch dtype -> XP_U8 for bytes and for one type of 8 bits, else -1, filled as types are met."""

    def __init__(self, own):
        self.own = own

    def __missing__(self, dtype):
        found = self[dtype] = XP_U8 if str(dtype) in ("torch.uint8", self.own) else -1
        return found


_types = _Types()
_codes, _scales = _Bytes("torch.float8_e4m3fn"), _Bytes("torch.float8_e8m0fnu")
_current_device = None   # asks torch for it, once torch is there


def _device_of(t) -> int:
    """The current device, as torch says; 0 where the tensors are not torch's."""
    global _current_device
    if _current_device is None:
        torch = sys.modules.get("torch")
        if torch is None:
            return 0
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


def _refuse_devices(tensors, current):
    at = sorted({t.get_device() for t in tensors if t is not None})
    raise ValueError(f"tensors on devices {at}, not all on the current one, {current} (-1: the host)")


def _refuse_matrix(t, shape, what, dtype, types):
    if t.shape != shape or types[t.dtype] != dtype:
        raise ValueError(f"{what} is {tuple(t.shape)} of {t.dtype}, not {tuple(shape)} of its type")
    raise ValueError(f"{what}'s columns are {t.stride()[1]} elements apart")


def _matrix(t, shape, what, dtype, device, types=_types):
    """(address, stride) of a matrix of a shape and type whose columns are side by side."""
    stride, step = t.stride()
    if t.shape != shape or (step != 1 and shape[1] > 1) or types[t.dtype] != dtype:
        _refuse_matrix(t, shape, what, dtype, types)
    if t.get_device() != device:
        _refuse_devices((t,), device)
    return t.data_ptr(), stride


def _vector(t, n, what, dtype, device):
    """The address of n contiguous elements (None: none)."""
    if t is None:
        return None
    if t.numel() != n or not t.is_contiguous() or _types[t.dtype] != dtype:
        raise ValueError(f"{what} is not {n} contiguous elements of its type")
    if t.get_device() != device:
        _refuse_devices((t,), device)
    return t.data_ptr()


def _block8(codes, scales, shape, block_rows, what, device):
    """(codes, stride, scales, stride) of a matrix in 8 bits; both or neither."""
    if codes is None or scales is None:
        if codes is not scales:
            raise ValueError(f"{what} without its scales, or scales without codes")
        return None, 0, None, 0
    rows, cols = shape
    if block_rows != 1:
        if block_rows != XP_BLOCK8:
            raise ValueError(f"{what}: blocks of {block_rows} rows, neither 1 nor 128")
        rows = (rows + 127) // 128
    p, s = _matrix(codes, shape, what, XP_U8, device, _codes)
    ps, ss = _matrix(scales, (rows, (cols + 127) // 128), "scales", XP_U8, device, _scales)
    return p, s, ps, ss


def _float(t, what):
    dt = _types[t.dtype]
    if dt == XP_U8:
        raise ValueError(f"{what} is {t.dtype}")
    return dt


def _check(st: int, where: str):
    if st != XP_OK:
        xp._check(st, where)


def xp_block8_encode(x, codes=None, scales=None, codes_t=None, scales_t=None, block_rows: int = 1, stream=None) -> None:
    """x (rows x cols) in 8 bits into codes and scales, and its transpose into codes_t and scales_t; either pair may be None."""
    shape, dt, dev = x.shape, _float(x, "x"), _device_of(x)
    rows, cols = shape
    px, sx = _matrix(x, shape, "x", dt, dev)
    pc, sc, ps, ss = _block8(codes, scales, shape, block_rows, "codes", dev)
    pct, sct, pst, sst = _block8(codes_t, scales_t, (cols, rows), block_rows, "codes_t", dev)
    st = _encode(px, sx, rows, cols, dt, block_rows, pc, sc, ps, ss, pct, sct, pst, sst, stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_block8_encode")


def xp_block8_decode(codes, scales, out, block_rows: int = 1, stream=None) -> None:
    """The values that a matrix in 8 bits stands for, into out."""
    shape, dt, dev = out.shape, _float(out, "out"), _device_of(out)
    rows, cols = shape
    po, so = _matrix(out, shape, "out", dt, dev)
    pc, sc, ps, ss = _block8(codes, scales, shape, block_rows, "codes", dev)
    st = _decode(pc, sc, ps, ss, rows, cols, block_rows, po, so, dt, stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_block8_decode")


def xp_matmul8(a, a_scales, b, b_scales, c, a_block_rows: int = 1, b_block_rows: int = 1, accumulate: bool = False, stream=None) -> None:
    """c = a b^T (accumulate: c + a b^T) of a (m x k) and b (n x k) in 8 bits."""
    shape, dt, dev = a.shape, _float(c, "c"), _device_of(c)
    (m, k), n = shape, b.shape[0]
    pa, sa, psa, ssa = _block8(a, a_scales, shape, a_block_rows, "a", dev)
    pb, sb, psb, ssb = _block8(b, b_scales, (n, k), b_block_rows, "b", dev)
    pc, sc = _matrix(c, (m, n), "c", dt, dev)
    st = _matmul(pa, sa, psa, ssa, a_block_rows, pb, sb, psb, ssb, b_block_rows, pc, sc, m, n, k, dt, 1 if accumulate else 0,
                 stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_matmul8")


def xp_matmul8_status() -> int:
    """Waits for the device; XP_ERR_TIMEOUT if a product ever gave up a wait, else XP_OK."""
    st = _lib.xp_matmul8_status()
    if st not in (XP_OK, xp.XP_ERR_TIMEOUT):
        xp._check(st, "xp_matmul8_status")
    return st


def xp_rmsnorm_forward(x, gamma, y=None, residual=None, added=None, rstd=None, y8=None, y8_scales=None, eps: float = 1e-5, stream=None) -> None:
    """The root-mean-square norm of x, or of x + residual (stored in added), into y, and in 8 bits into y8."""
    shape, dt, dev = x.shape, _float(x, "x"), _device_of(x)
    rows, cols = shape
    wdt = dt if gamma is None else _float(gamma, "gamma")
    px, sx = _matrix(x, shape, "x", dt, dev)
    pr, sr = (None, 0) if residual is None else _matrix(residual, shape, "residual", dt, dev)
    pa, sa = (None, 0) if added is None else _matrix(added, shape, "added", dt, dev)
    py, sy = (None, 0) if y is None else _matrix(y, shape, "y", dt, dev)
    p8, s8, p8s, s8s = _block8(y8, y8_scales, shape, 1, "y8", dev)
    st = _forward(px, sx, pr, sr, _vector(gamma, cols, "gamma", wdt, dev), pa, sa, py, sy, p8, s8, p8s, s8s,
                  _vector(rstd, rows, "rstd", XP_F32, dev), rows, cols, eps, dt, wdt, stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_rmsnorm_forward")


def xp_rmsnorm_workspace(rows: int, cols: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.xp_rmsnorm_workspace(rows, cols, ctypes.byref(out)), "xp_rmsnorm_workspace")
    return out.value


def xp_rmsnorm_backward(dy, h, gamma, rstd, dx, dgamma=None, workspace=None, dadded=None, accumulate: bool = False, stream=None) -> None:
    """dx (+ dadded), and over the rows dgamma, from dy, the norm's input h and the forward pass's rstd."""
    shape, dt, dev = h.shape, _float(h, "h"), _device_of(h)
    rows, cols = shape
    wdt = dt if gamma is None else _float(gamma, "gamma")
    work, nbytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace is not contiguous")
        if workspace.get_device() != dev:
            _refuse_devices((workspace,), dev)
        work, nbytes = workspace.data_ptr(), workspace.nbytes
    pdy, sdy = _matrix(dy, shape, "dy", dt, dev)
    ph, sh = _matrix(h, shape, "h", dt, dev)
    pa, sa = (None, 0) if dadded is None else _matrix(dadded, shape, "dadded", dt, dev)
    pdx, sdx = _matrix(dx, shape, "dx", dt, dev)
    st = _backward(pdy, sdy, ph, sh, _vector(gamma, cols, "gamma", wdt, dev), _vector(rstd, rows, "rstd", XP_F32, dev), pa, sa, pdx, sdx,
                   _vector(dgamma, cols, "dgamma", XP_F32, dev), rows, cols, dt, wdt, 1 if accumulate else 0, work, nbytes,
                   stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_rmsnorm_backward")


def _top(ids, teacher, rows, dev):
    """(ids, teacher, entries per row), both rows x top side by side."""
    shape = ids.shape
    if shape[0] != rows or str(ids.dtype) != "torch.int32" or not ids.is_contiguous():
        raise ValueError(f"ids is {tuple(shape)} of {ids.dtype}, not {rows} contiguous rows of torch.int32")
    if teacher.shape != shape:
        raise ValueError(f"teacher is {tuple(teacher.shape)}, not {tuple(shape)}")
    if ids.get_device() != dev:
        _refuse_devices((ids,), dev)
    return ids.data_ptr(), _vector(teacher, rows * shape[1], "teacher", XP_F32, dev), shape[1]


def xp_distill_forward(logits, ids, teacher, loss, lse=None, temperature: float = 1.0, stream=None) -> None:
    """Each row's loss against the teacher's logits (rows x top, fp32) at ids (int32), and the row's log-sum-exp."""
    shape, dt, dev = logits.shape, _float(logits, "logits"), _device_of(logits)
    rows, vocab = shape
    pi, pt, top = _top(ids, teacher, rows, dev)
    pz, sz = _matrix(logits, shape, "logits", dt, dev)
    st = _distill(pz, sz, pi, pt, rows, vocab, top, temperature, _vector(loss, rows, "loss", XP_F32, dev), _vector(lse, rows, "lse", XP_F32, dev), dt,
                  stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_distill_forward")


def xp_distill_backward(logits, ids, teacher, lse, dloss, dlogits, temperature: float = 1.0, stream=None) -> None:
    """dlogits from dloss (one per row) and the forward pass's lse; dlogits may be logits."""
    shape, dt, dev = logits.shape, _float(logits, "logits"), _device_of(logits)
    rows, vocab = shape
    pi, pt, top = _top(ids, teacher, rows, dev)
    pz, sz = _matrix(logits, shape, "logits", dt, dev)
    pd, sd = _matrix(dlogits, shape, "dlogits", dt, dev)
    st = _distill_back(pz, sz, pi, pt, _vector(lse, rows, "lse", XP_F32, dev), _vector(dloss, rows, "dloss", XP_F32, dev), rows, vocab, top,
                       temperature, pd, sd, dt, stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_distill_backward")

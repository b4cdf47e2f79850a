"""ctypes binding of the training operators of libxp.so (include/xp_train.h): same names, argument marshalling only.

Tensors are torch tensors (or objects with the same `data_ptr()`, `shape`, `stride()` and `dtype`): their pointers,
sizes, strides and types are read off, and shapes that do not belong together raise ValueError before the call.
Streams, and the errors of the library itself (`XpError`), are as in `xp`.
"""
from __future__ import annotations

import ctypes

from . import xp
from .xp import XP_BF16, XP_F32, XP_OK, XP_U8, XpError, _stream  # noqa: F401

XP_LAYERNORM_MAX_COLS = 131072
XP_LAYERNORM_MAX_ROWS = 1 << 28
XP_STATE8_BLOCK = 32
XP_GROUP_MAX_ELEMENTS = 1 << 40
XP_GROUP_MAX_STEP = 1 << 52
XP_ADAMW_SKIP_NONFINITE = 1

# every entry point include/xp_train.h declares
EXPORTS = [
    "xp_layernorm_forward", "xp_layernorm_workspace", "xp_layernorm_backward", "xp_group_create", "xp_group_destroy",
    "xp_group_set_grads", "xp_group_set_step", "xp_group_get_step", "xp_grad_norm", "xp_adamw_step", "xp_state8_decode",
]


class xp_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("count", ctypes.c_size_t), ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)]


class xp_group_config(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
                ("seed", ctypes.c_uint32), ("step", ctypes.c_uint64)]


class xp_grad_report(ctypes.Structure):
    _fields_ = [("sumsq", ctypes.c_double), ("norm", ctypes.c_float), ("scale", ctypes.c_float),
                ("nonfinite", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]


_lib = xp._lib
_P, _I, _Z, _F, _U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_uint64
for _name, _args in {
    "xp_layernorm_forward": [_P, _Z, _P, _P, _P, _Z, _P, _P, _Z, _Z, _F, _I, _I, _P],
    "xp_layernorm_workspace": [_Z, _Z, ctypes.POINTER(_Z)],
    "xp_layernorm_backward": [_P, _Z, _P, _Z, _P, _P, _P, _P, _Z, _P, _P, _Z, _Z, _I, _I, _I, _P, _Z, _P],
    "xp_group_create": [ctypes.POINTER(xp_group_config), _I, ctypes.POINTER(xp_tensor), ctypes.POINTER(_P)],
    "xp_group_destroy": [_P],
    "xp_group_set_grads": [_P, ctypes.POINTER(_P), _P],
    "xp_group_set_step": [_P, _U64, _P],
    "xp_group_get_step": [_P, ctypes.POINTER(_U64), _P],
    "xp_grad_norm": [_P, _F, _F, _I, _P, _P],
    "xp_adamw_step": [_P, _F, _P, _F, _P, _I, _P],
    "xp_state8_decode": [_P, _P, _P, _P, _Z, _P, _P, _I, _P],
}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = ctypes.c_int
_forward, _backward, _norm, _step, _decode = (_lib.xp_layernorm_forward, _lib.xp_layernorm_backward, _lib.xp_grad_norm,
                                              _lib.xp_adamw_step, _lib.xp_state8_decode)

_DTYPES = {"torch.float32": XP_F32, "torch.bfloat16": XP_BF16, "torch.uint8": XP_U8}
_types = {}   # torch dtype -> xp_dtype, filled as types are met
_REPORT_BYTES = ctypes.sizeof(xp_grad_report)
_gradients = {}   # group -> (its tensors' lengths, their gradients' type)


def _dtype(t) -> int:
    found = _types.get(t.dtype)
    if found is None:
        if str(t.dtype) not in _DTYPES:
            raise ValueError(f"no xp_dtype for {t.dtype}")
        found = _types[t.dtype] = _DTYPES[str(t.dtype)]
    return found


def _check(st: int, where: str):
    if st != XP_OK:
        xp._check(st, where)


def _refuse_rows(named, shape, dtype):
    """Says which of several matrices does not have the first one's shape and type, or its columns side by side."""
    for what, t in named:
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{what} is {tuple(t.shape)} of {t.dtype}, not {tuple(shape)} of {dtype}")
        if shape[1] > 1 and t.stride()[1] != 1:
            raise ValueError(f"{what}'s columns are {t.stride()[1]} elements apart")


def _vector(t, n, what, dtype):
    """The address of n contiguous elements (None: none)."""
    if t is None:
        return None
    if t.numel() != n or not t.is_contiguous() or _types.get(t.dtype) != dtype and _dtype(t) != dtype:
        raise ValueError(f"{what} is not {n} contiguous elements of its type")
    return t.data_ptr()


def _report(t):
    """The address of an xp_grad_report's 32 bytes.  (One that is not 16-byte aligned is for the library to refuse.)"""
    p = t.data_ptr()
    if (t.nbytes < _REPORT_BYTES or not t.is_contiguous()) and p & 15 == 0:
        raise ValueError(f"report is not {_REPORT_BYTES} contiguous bytes")
    return p


def xp_layernorm_forward(x, gamma, beta, y, mean=None, rstd=None, eps: float = 1e-5, stream=None) -> None:
    """y = layer norm of each row of x (rows x cols), with its statistics where mean and rstd are given."""
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    (xs, xc), (ys, yc) = x.stride(), y.stride()
    if y.shape != shape or y.dtype != dtype or (xc != 1 or yc != 1) and cols > 1:
        _refuse_rows((("x", x), ("y", y)), shape, dtype)
    dt = _types.get(dtype) or _dtype(x)
    wdt = _dtype(gamma) if gamma is not None else dt if beta is None else _dtype(beta)
    st = _forward(x.data_ptr(), xs, _vector(gamma, cols, "gamma", wdt), _vector(beta, cols, "beta", wdt), y.data_ptr(), ys,
                  _vector(mean, rows, "mean", XP_F32), _vector(rstd, rows, "rstd", XP_F32), rows, cols, eps, dt, wdt,
                  stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_layernorm_forward")


def xp_layernorm_workspace(rows: int, cols: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.xp_layernorm_workspace(rows, cols, ctypes.byref(out)), "xp_layernorm_workspace")
    return out.value


def xp_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, workspace=None, accumulate: bool = False,
                          stream=None) -> None:
    """dx, and over the rows dgamma and dbeta, from dy and what the forward pass gave."""
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    (dys, dyc), (xs, xc), (dxs, dxc) = dy.stride(), x.stride(), dx.stride()
    if (dy.shape != shape or dx.shape != shape or dy.dtype != dtype or dx.dtype != dtype
            or (dyc != 1 or xc != 1 or dxc != 1) and cols > 1):
        _refuse_rows((("dy", dy), ("x", x), ("dx", dx)), shape, dtype)
    dt = _types.get(dtype) or _dtype(x)
    wdt = dt if gamma is None else _dtype(gamma)
    work, nbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    if work is not None and not workspace.is_contiguous():
        raise ValueError("workspace is not contiguous")
    st = _backward(dy.data_ptr(), dys, x.data_ptr(), xs, _vector(gamma, cols, "gamma", wdt), _vector(mean, rows, "mean", XP_F32),
                   _vector(rstd, rows, "rstd", XP_F32), dx.data_ptr(), dxs, _vector(dgamma, cols, "dgamma", XP_F32),
                   _vector(dbeta, cols, "dbeta", XP_F32), rows, cols, dt, wdt, 1 if accumulate else 0, work, nbytes,
                   stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_layernorm_backward")


def xp_group_create(params, grads, m=None, v=None, *, m_scales=None, v_scales=None, copies=None, weight_decay=0.0,
                    beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, seed: int = 0, step: int = 0) -> int:
    """A group of tensors: lists of the same length.  params None: a group for xp_grad_norm alone.  States of
    torch.uint8 are 8-bit codes and need scales; weight_decay is one number or a list.  The caller keeps the
    tensors alive as long as the group."""
    n = len(grads)
    decay = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * n
    named = {"param": params, "m": m, "v": v, "m_scale": m_scales, "v_scale": v_scales, "copy": copies}
    cfg = xp_group_config(beta1=beta1, beta2=beta2, eps=eps, seed=seed, step=step, grad_dtype=_dtype(grads[0]) if n else XP_F32,
                          param_dtype=_dtype(params[0]) if params else XP_F32, state_dtype=_dtype(m[0]) if m else XP_F32)
    if len(decay) != n or any(x is not None and len(x) != n for x in named.values()):
        raise ValueError("the lists differ in length")
    want = {"param": cfg.param_dtype, "grad": cfg.grad_dtype, "m": cfg.state_dtype, "v": cfg.state_dtype, "copy": XP_BF16,
            "m_scale": XP_U8, "v_scale": XP_U8}
    named["grad"] = grads
    counts = [t.numel() for t in grads]
    blocks = [-(-c // XP_STATE8_BLOCK) for c in counts]
    columns = {}
    for name, tensors in named.items():
        sizes, dtype = blocks if name.endswith("scale") else counts, want[name]
        columns[name] = [None] * n if tensors is None else [_vector(t, k, f"{name} {i}", dtype) for i, (t, k) in enumerate(zip(tensors, sizes))]
    rows = zip(columns["param"], columns["grad"], columns["m"], columns["v"], columns["m_scale"], columns["v_scale"], columns["copy"],
               counts, decay)
    table = (xp_tensor * max(n, 1))(*[xp_tensor(*row) for row in rows])
    out = ctypes.c_void_p()
    _check(_lib.xp_group_create(ctypes.byref(cfg), n, table, ctypes.byref(out)), "xp_group_create")
    _gradients[out.value] = counts, grads[0].dtype
    return out.value


def xp_group_destroy(group: int) -> None:
    _gradients.pop(group, None)
    _check(_lib.xp_group_destroy(group), "xp_group_destroy")


def xp_group_set_grads(group: int, grads, stream=None) -> None:
    """Other gradient buffers, of the lengths and type the group was made with."""
    if group not in _gradients:
        raise ValueError("not a group that xp_group_create made")
    counts, dtype = _gradients[group]
    if len(grads) != len(counts):
        raise ValueError(f"{len(grads)} gradients for {len(counts)} tensors")
    if not all([t.numel() == n and t.dtype == dtype and t.is_contiguous() for t, n in zip(grads, counts)]):
        for i, (t, n) in enumerate(zip(grads, counts)):
            _vector(t, n, f"grad {i}", _types[dtype])
    ptrs = (ctypes.c_void_p * len(counts))(*[t.data_ptr() for t in grads])
    _check(_lib.xp_group_set_grads(group, ptrs, _stream(stream)), "xp_group_set_grads")


def xp_group_set_step(group: int, step: int, stream=None) -> None:
    _check(_lib.xp_group_set_step(group, step, _stream(stream)), "xp_group_set_step")


def xp_group_get_step(group: int, stream=None) -> int:
    out = ctypes.c_uint64()
    _check(_lib.xp_group_get_step(group, ctypes.byref(out), _stream(stream)), "xp_group_get_step")
    return out.value


def xp_grad_norm(group: int, report, grad_scale: float = 1.0, max_norm: float = 0.0, accumulate: bool = False, stream=None) -> None:
    """The norm of the group's gradients into `report`, 32 bytes of device memory laid out as xp_grad_report."""
    _check(_norm(group, grad_scale, max_norm, 1 if accumulate else 0, _report(report), stream if stream is None else _stream(stream)),
           "xp_grad_norm")


def xp_adamw_step(group: int, lr: float, report=None, grad_scale: float = 1.0, skip_nonfinite: bool = False, lr_dev=None,
                  stream=None) -> None:
    """One AdamW step on the group's tensors, gradients scaled by the report's scale if there is one; the rate is lr_dev's
    first element if there is one."""
    if lr_dev is not None and (lr_dev.numel() < 1 or _dtype(lr_dev) != XP_F32):
        raise ValueError("lr_dev is not an fp32 number")
    _check(_step(group, lr, None if lr_dev is None else lr_dev.data_ptr(), grad_scale, None if report is None else _report(report),
                 XP_ADAMW_SKIP_NONFINITE if skip_nonfinite else 0, stream if stream is None else _stream(stream)), "xp_adamw_step")


def xp_state8_decode(m, m_scale, v, v_scale, m_out, v_out, stream=None) -> None:
    """The values of 8-bit states, m's into m_out and v's into v_out (either may be None)."""
    out = m_out if m_out is not None else v_out
    if out is None:
        return
    count, dt = out.numel(), _dtype(out)
    blocks = -(-count // XP_STATE8_BLOCK)
    pm = pms = pmo = pv = pvs = pvo = None
    if m_out is not None:
        pm, pms, pmo = _vector(m, count, "m", XP_U8), _vector(m_scale, blocks, "m_scale", XP_U8), _vector(m_out, count, "m_out", dt)
    if v_out is not None:
        pv, pvs, pvo = _vector(v, count, "v", XP_U8), _vector(v_scale, blocks, "v_scale", XP_U8), _vector(v_out, count, "v_out", dt)
    st = _decode(pm, pms, pv, pvs, count, pmo, pvo, dt, stream if stream is None else _stream(stream))
    if st:
        xp._check(st, "xp_state8_decode")

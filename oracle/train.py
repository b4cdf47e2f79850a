"""The training operators by their formulas, in numpy: layer norm forward and backward, the gradient norm, the AdamW
step and the 8-bit states' codes.

Written from the formulas alone, for arrays of any float type: in float64 they are the values the kernels'
results are near to, in float32 every operation is rounded as IEEE says, in the order stated here."""
from __future__ import annotations

import numpy as np

BLOCK = 32


def layernorm_forward(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) of each row of x."""
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) of the sum of dy * y, through mean and rstd."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    a = dy if gamma is None else dy * gamma
    dx = (a - a.mean(1, keepdims=True) - xhat * (a * xhat).mean(1, keepdims=True)) * rstd[:, None]
    return dx, (dy * xhat).sum(0), dy.sum(0)


def grad_norm(grads, grad_scale=1.0, max_norm=0.0):
    """(sum of squares, norm, scale) of all arrays as one vector."""
    sumsq = float(sum(np.sum(np.asarray(g, np.float64) ** 2) for g in grads))
    norm = grad_scale * np.sqrt(sumsq)
    return sumsq, norm, grad_scale * (max_norm / norm if 0 < max_norm < norm else 1.0)


def adamw(p, g, m, v, t, lr, decay, beta1=0.9, beta2=0.999, eps=1e-8, scale=1.0):
    """(p, m, v) after step t (the first is 1).  In float32 every constant is the one the header's formulas give,
    rounded, and each operation rounds."""
    f = p.dtype.type
    g = g.astype(p.dtype) * f(scale)
    m = m * f(beta1) + g * f(1 - beta1)
    v = v * f(beta2) + g * f(1 - beta2) * g
    alpha = f(lr) * f(1 / (1 - beta1 ** t))
    rs = f(1 / np.sqrt(1 - beta2 ** t))
    keep = f(1) - f(lr) * f(decay)
    p = p * keep - (m * alpha) / (np.sqrt(v) * rs + f(eps))
    return p, m, v


# ---- 8-bit states

def _mix(x):
    x = ((x ^ (x >> 16)) * 0xDDF15BA9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xE31B8755) & 0xFFFFFFFF
    return x ^ (x >> 16)


def rounding_bits(seed, t, pos):
    """The 16-bit hashes that round m and v at the positions `pos` (python integers or uint64) in step t."""
    key = _mix((seed * 0x8ED88009 + _mix(t & 0xFFFFFFFF)) & 0xFFFFFFFF)
    h = np.array([_mix((int(i) % (1 << 32) * 0x8ED88009 + (int(i) >> 32) * 0xB86D3E2F + key) & 0xFFFFFFFF) for i in pos], np.uint32)
    return h >> np.uint32(16), h & np.uint32(0xFFFF)


def _blocks(x):
    n = len(x)
    return np.concatenate([x, np.zeros(-n % BLOCK, x.dtype)]).reshape(-1, BLOCK)


def encode(x, hash16, signed):
    """(codes, scales) of float32 values: x's pattern plus 16 h + 8, cut to an exponent and 3 mantissa bits, relative
    to the block's largest exponent."""
    n = len(x)
    bits = _blocks(np.abs(x).astype(np.float32)).view(np.uint32)
    e = (bits >> 23).max(1)
    cut = ((bits.astype(np.int64) + _blocks(hash16.astype(np.int64) * 16 + 8)) >> 20) - (8 * e.astype(np.int64) - (119 if signed else 247))[:, None]
    c = np.where(bits == 0, 0, np.clip(cut, 0 if signed else 1, 127 if signed else 255))
    if signed:
        c = c + 128 * ((c > 0) & (_blocks(x) < 0))
    return c.reshape(-1)[:n].astype(np.uint8), e.astype(np.uint8)


def decode(code, scale, signed):
    """The values that codes stand for, in float64: 2^(E - 127) times powers of 2 below it, 8 codes to each."""
    n = len(code)
    c = _blocks(code.astype(np.int64))
    mag = c % 128 if signed else c
    at = np.maximum(mag + 8 * scale.astype(np.int64)[:, None] - (119 if signed else 247), 0)   # below the least pattern: 0
    with np.errstate(over="ignore"):
        x = np.where(mag == 0, 0.0, np.ldexp(1 + (at % 8) / 8, at // 8 - 127))
    x = np.where(at < 8, at * 2.0 ** -129 * (mag > 0), x)        # patterns without an exponent are subnormal numbers
    x = np.where(signed & (c >= 128), -x, x)
    return np.where(scale[:, None] == 255, np.nan, x).reshape(-1)[:n]

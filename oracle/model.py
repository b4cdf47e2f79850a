"""The operators of a layer in 8 bits by their formulas, in numpy and float64: encoding by blocks of 128 and decoding, the
product, the root-mean-square norm forward and backward, distillation from a teacher's top logits forward and backward.

Written from the formulas alone; a matrix in 8 bits is (codes, scales), uint8 arrays."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def code_values():
    """The 256 codes' values: a sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, f = c >> 3 & 15, c & 7
    mag = np.where(e == 0, f * 2.0 ** -9, np.ldexp(8.0 + f, e - 10))
    mag[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -mag, mag)


_POSITIVE = code_values()[:127]                            # ascending: codes 0 .. 126
_MIDDLES = (_POSITIVE[1:] + _POSITIVE[:-1]) / 2


def nearest_code(x):
    """The nearest code of each value (448 at most in magnitude, by rounding), ties to the even code."""
    mag = np.abs(x)
    lower = np.searchsorted(_MIDDLES, mag, side="left")    # the first middle that is not below: at one, the lower code
    tie = (lower < len(_MIDDLES)) & (mag == _MIDDLES[np.minimum(lower, len(_MIDDLES) - 1)])
    c = np.where(tie & (lower % 2 == 1), lower + 1, lower)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def scale_of(top):
    """The least E of 0 .. 254 with top <= 448 * 2^(E - 127); 255 where top is not finite."""
    with np.errstate(divide="ignore", invalid="ignore"):
        m, p = np.frexp(np.asarray(top, np.float64))        # top = m 2^p, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = np.maximum(p - 9 + (m > 0.875) + 127, 0)
    return np.where(np.isfinite(top), np.where(np.asarray(top) == 0, 0, e), 255).astype(np.uint8)


def _blocks(x, block_rows):
    """Blocks of rows, rows, blocks of columns, columns; zeros past the edges."""
    r, c = x.shape
    x = np.pad(x, ((0, -r % block_rows), (0, -c % BLOCK)))
    return x.reshape(x.shape[0] // block_rows, block_rows, -1, BLOCK)


def encode(x, block_rows=1):
    """(codes, scales) of a matrix."""
    r, c = x.shape
    b = _blocks(np.asarray(x, np.float64), block_rows)
    e = scale_of(np.abs(b).max((1, 3)))
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.ldexp(b, 127 - e.astype(np.int64)[:, None, :, None])
        codes = np.where((e == 255)[:, None, :, None], 0x7F, nearest_code(np.where(np.isfinite(y), y, 0)))
    return codes.reshape(-1, codes.shape[2] * BLOCK)[:r, :c].astype(np.uint8), e


def decode(codes, scales, block_rows=1):
    r, c = codes.shape
    e = np.repeat(np.repeat(scales.astype(np.int64), block_rows, 0)[:r], BLOCK, 1)[:, :c]
    return np.where(e == 255, np.nan, np.ldexp(code_values()[codes], e - 127))


def product(a, a_scales, b, b_scales, a_block_rows=1, b_block_rows=1):
    """(a b^T, the sums of the products' magnitudes)."""
    x, y = decode(a, a_scales, a_block_rows), decode(b, b_scales, b_block_rows)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def rmsnorm_forward(h, gamma=None, eps=1e-5):
    """(y, rstd) of each row of h."""
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if gamma is None else y * gamma), rstd


def rmsnorm_backward(dy, h, gamma, rstd, dadded=None):
    """(dx, dgamma) of the sum of dy * y, through rstd, and of dadded * h."""
    xhat = h * rstd[:, None]
    a = dy if gamma is None else dy * gamma
    dx = (a - xhat * (a * xhat).mean(1, keepdims=True)) * rstd[:, None]
    return (dx if dadded is None else dx + dadded), (dy * xhat).sum(0)


def teacher(ids, t, vocab, temperature):
    """(p, where an entry counts) of each row's entries; p is 0 in rows without any."""
    there = (ids >= 0) & (ids < vocab) & (t != -np.inf)
    p = np.zeros(t.shape)
    for i in range(len(t)):
        u = t[i, there[i]] / temperature
        if len(u):
            w = np.exp(u - u.max())
            p[i, there[i]] = w / w.sum()
    return p, there


def distill_forward(z, ids, t, temperature=1.0):
    """(loss, lse) of each row; both 0 in rows without entries, whatever their logits."""
    p, there = teacher(ids, t, z.shape[1], temperature)
    loss, lse = np.zeros(len(z)), np.zeros(len(z))
    for i in range(len(z)):
        if not there[i].any():
            continue
        s = z[i] / temperature
        with np.errstate(invalid="ignore"):
            lse[i] = s.max() + np.log(np.exp(s - s.max()).sum())
        q, logq = p[i, there[i]], s[ids[i, there[i]]] - lse[i]
        some = q > 0
        loss[i] = temperature ** 2 * (q[some] * (np.log(q[some]) - logq[some])).sum()
    return loss, lse


def distill_backward(z, ids, t, lse, dloss, temperature=1.0):
    p, there = teacher(ids, t, z.shape[1], temperature)
    d = np.zeros(z.shape)
    for i in range(len(z)):
        if there[i].any():
            d[i] = np.exp(z[i] / temperature - lse[i])
            np.subtract.at(d[i], ids[i, there[i]], p[i, there[i]])
    return d * (dloss * temperature)[:, None]

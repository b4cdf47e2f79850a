"""The operators of a layer in 8 bits on the GPU against their formulas in 64 bits (oracle.model): codes and scales bit for
bit, products of whole numbers exactly, everything else within bounds that follow from rounding.

U = 2^-24 is fp32's rounding error, a power of 2 is off by at most 2^-22 relatively (two units in the last place of the
hardware's approximation).  A sum of n terms that is made in a chain of c additions and a tree above it is off by at most
(c + tree) U times the sum of magnitudes."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import model
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
POW = 2.0 ** -22


@pytest.fixture(scope="module")
def xm():
    torch_cuda()
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_model as xm
    return xm


@pytest.fixture(autouse=True)
def no_waits_given_up(xm):
    yield
    assert xm.xp_matmul8_status() == xm.XP_OK


def _type(torch, name):
    """The type, and what rounding to it may be off relatively."""
    return {"f32": (torch.float32, U), "bf16": (torch.bfloat16, 2.0 ** -8)}[name]


def _f64(t):
    return t.double().cpu().numpy()


def _matrix(torch, rows, cols, dtype, pad=0, offset=0, fill=None, values=None):
    """A rows x cols view whose rows are pad elements further apart and whose first element is `offset` elements into its
    buffer, and the buffer; what is between holds `fill` (NaN)."""
    fill = float("nan") if fill is None else fill
    buf = torch.full((offset + rows * (cols + pad) + 16,), fill, dtype=dtype, device="cuda")
    m = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if values is not None:
        m.copy_(torch.as_tensor(values).to(dtype))
    return m, buf


def _bytes(torch, rows, cols, step=16, fill=0x7F):
    """A matrix of bytes whose rows are a multiple of `step` apart, and one more: what is between holds `fill`."""
    pitch = (cols + step - 1) // step * step + step
    return torch.full((rows, pitch), fill, dtype=torch.uint8, device="cuda")[:, :cols]


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- encoding

ENCODED = [(1, 1), (1, 128), (3, 5), (2, 129), (127, 3), (128, 128), (129, 127), (130, 260), (256, 384), (257, 1001), (64, 4100), (1000, 132)]


def _spread(rows, cols, seed):
    """Values of every magnitude, block by block and element by element, with zeros of both signs."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 4, (rows, cols)))
    x *= np.exp2(rng.integers(-100, 100, (rows, 1))) * np.exp2(rng.integers(-20, 20, (1, cols)))
    x[rng.random((rows, cols)) < 0.02] = 0.0
    x[rng.random((rows, cols)) < 0.02] = -0.0
    return x


def _check_encode(torch, xm, x, block_rows, which="both", out_step=16):
    rows, cols = x.shape
    x64 = _f64(x)
    codes, scales = (_bytes(torch, rows, cols, out_step), _bytes(torch, _ceil(rows, block_rows), _ceil(cols, 128), 4)) if which != "t" else (None, None)
    codes_t, scales_t = (_bytes(torch, cols, rows, out_step), _bytes(torch, _ceil(cols, block_rows), _ceil(rows, 128), 4)) if which != "plain" else (None, None)
    xm.xp_block8_encode(x, codes, scales, codes_t, scales_t, block_rows=block_rows)
    for c, s, want in ((codes, scales, x64), (codes_t, scales_t, x64.T)):
        if c is None:
            continue
        want_c, want_s = model.encode(want, block_rows)
        assert np.array_equal(s.cpu().numpy(), want_s), (rows, cols, block_rows)
        assert np.array_equal(c.cpu().numpy(), want_c), (rows, cols, block_rows)
        for t in (c, s):   # nothing between the rows is written
            assert (t._base[:, t.shape[1]:] == 0x7F).all()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", ENCODED)
def test_encode(xm, rows, cols, name, block_rows):
    torch = torch_cuda()
    dtype, _ = _type(torch, name)
    x, _ = _matrix(torch, rows, cols, dtype, values=_spread(rows, cols, rows + cols))
    for which in ("both", "plain", "t"):
        _check_encode(torch, xm, x, block_rows, which)


@pytest.mark.parametrize("pad,offset,step", [(4, 0, 16), (1, 0, 16), (0, 1, 16), (3, 2, 16), (0, 0, 1), (8, 8, 4)])
@pytest.mark.parametrize("rows,cols", [(130, 256), (257, 300)])
def test_encode_strides_and_alignment(xm, rows, cols, pad, offset, step):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        x, _ = _matrix(torch, rows, cols, _type(torch, name)[0], pad, offset, values=_spread(rows, cols, 7))
        _check_encode(torch, xm, x, 1, out_step=step)
        _check_encode(torch, xm, x, 128, out_step=step)


@pytest.mark.parametrize("rows,cols", [(1, 513), (2, 512), (5, 515), (130, 640), (131, 1031), (3, 2049)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (0, 2), (0, 3), (1, 0), (2, 1), (3, 3), (4, 2)])
def test_encode_rows_that_begin_anywhere(xm, rows, cols, pad, offset):
    # NaN lies around the matrix and between its rows
    torch = torch_cuda()
    x, _ = _matrix(torch, rows, cols, torch.bfloat16, pad, offset, values=_spread(rows, cols, 11))
    _check_encode(torch, xm, x, 1)
    _check_encode(torch, xm, x, 128, "plain")


def test_encode_where_it_is_decided(xm):
    # largest magnitudes at, below and above 448 times every power of two; elements at the middles between codes
    torch = torch_cuda()
    tops = np.concatenate([[448 * 2.0 ** e, np.nextafter(np.float32(448 * 2.0 ** e), np.float32(np.inf)), 256 * 2.0 ** e, 2.0 ** e] for e in range(-133, 119)])
    middles = np.concatenate([(model.code_values()[:126] + model.code_values()[1:127]) / 2, [0.0]])
    x = np.zeros((len(tops), 128))
    power = 2.0 ** (model.scale_of(tops.astype(np.float32)).astype(np.int64) - 127)
    x[:, 1:] = middles[None, :] * power[:, None] * np.where(np.arange(127) % 2, 1, -1)
    x = np.where(np.abs(x) > tops[:, None], 0, x)
    x[:, 0] = tops
    _check_encode(torch, xm, torch.from_numpy(x.astype(np.float32)).cuda(), 1, "plain")
    _check_encode(torch, xm, torch.from_numpy(x.astype(np.float32)).cuda(), 128)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_encode_blocks_that_are_not_finite(xm, name, value):
    torch = torch_cuda()
    x, _ = _matrix(torch, 260, 300, _type(torch, name)[0], values=_spread(260, 300, 3))
    x[5, 7] = x[140, 299] = x[259, 0] = value
    x[6, 130] = -value
    for block_rows in (1, 128):
        _check_encode(torch, xm, x, block_rows)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_decode_every_code_and_scale(xm, name):
    torch = torch_cuda()
    dtype, _ = _type(torch, name)
    codes, scales = _bytes(torch, 256, 256), _bytes(torch, 256, 2, 4)
    codes.copy_(torch.arange(256, dtype=torch.uint8).expand(256, 256))
    scales.copy_(torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 2))
    out = torch.empty(256, 256, dtype=dtype, device="cuda")
    xm.xp_block8_decode(codes, scales, out)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(model.decode(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)).to(dtype)
    assert np.array_equal(_f64(out), want.double().numpy(), equal_nan=True)


@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 130, 0, 0), (200, 1100, 0, 0), (130, 2048, 8, 8), (129, 1031, 3, 1), (5, 4096, 1, 0), (70, 520, 4, 4)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_decode_shapes(xm, rows, cols, pad, offset, block_rows):
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    c, s = rng.integers(0, 256, (rows, cols), dtype=np.uint8), rng.integers(90, 160, (_ceil(rows, block_rows), _ceil(cols, 128)), dtype=np.uint8)
    codes, scales = _bytes(torch, rows, cols, 1 if offset else 16), _bytes(torch, *s.shape, 1)
    codes.copy_(torch.from_numpy(c))
    scales.copy_(torch.from_numpy(s))
    want = model.decode(c, s, block_rows)
    for name in ("f32", "bf16"):
        out, buf = _matrix(torch, rows, cols, _type(torch, name)[0], pad, offset, fill=5.0)
        xm.xp_block8_decode(codes, scales, out, block_rows=block_rows)
        assert np.array_equal(_f64(out), want, equal_nan=True)
        if pad:
            assert (buf[offset:offset + rows * (cols + pad)].view(rows, -1)[:, cols:] == 5).all()


@pytest.mark.parametrize("rows,cols,pad,offset", [(100, 64, 0, 0), (100, 65, 0, 0), (20, 256, 8, 0), (20, 257, 0, 0), (9, 264, 0, 0), (9, 1279, 1, 0), (9, 1280, 1, 1), (9, 1281, 0, 3), (9, 1280, 0, 0)])
def test_decode_short_rows(xm, rows, cols, pad, offset):
    test_decode_shapes(xm, rows, cols, pad, offset, 1)


# ---------------------------------------------------------------- products

def _whole(torch, rows, cols, block_rows, seed, low=126, high=130):
    """Codes of whole numbers from -2 to 2 with scales 1/2 to 4: products are multiples of 1/4 and sums of up to 65536 of
    them are exact in fp32, in any order.  Between the rows lie NaN codes and scales."""
    rng = np.random.default_rng(seed)
    values = np.array([0x00, 0x38, 0x40, 0xB8, 0xC0, 0x80], np.uint8)      # 0, 1, 2, -1, -2, -0
    c = values[rng.integers(0, 6, (rows, cols))]
    s = rng.integers(low, high, (_ceil(rows, block_rows), _ceil(cols, 128)), dtype=np.uint8)
    codes, scales = _bytes(torch, rows, cols), _bytes(torch, *s.shape, 4, 0xFF)
    codes.copy_(torch.from_numpy(c))
    scales.copy_(torch.from_numpy(s))
    return codes, scales


def _values(torch, codes, scales, block_rows):
    return torch.from_numpy(model.decode(codes.cpu().numpy(), scales.cpu().numpy(), block_rows)).cuda()


# few rows; a tile's edges; rows and columns of every choice of tile, alone, shared by a cluster, and in pairs
PRODUCTS = [(1, 1, 1), (1, 5, 16), (2, 128, 128), (3, 129, 127), (16, 128, 129), (17, 300, 640), (33, 127, 1000), (64, 4096, 1024), (65, 257, 2100), (1, 4096, 4096),
            (1, 300, 9000), (100, 64, 5000), (128, 4096, 512), (129, 255, 300), (200, 1000, 3000), (256, 256, 128), (255, 4100, 1024), (300, 300, 300), (512, 4096, 260),
            (513, 2049, 385), (700, 5000, 130), (1025, 4096, 256), (1500, 9000, 140), (2000, 700, 2001), (3001, 2050, 4100), (5000, 33, 700), (16, 9000, 33), (1, 20001, 257)]


# Many rows, whose tiles pairs of CTAs and clusters of two pairs make, with each number of rows in a tile.
PRODUCTS += [(2596, 138, 228), (6920, 1, 397), (7319, 131, 356), (3240, 6325, 50), (4489, 5617, 90), (6978, 8031, 20), (5886, 569, 903), (148, 1948, 257),
             (943, 8118, 2134), (813, 6767, 2216), (6863, 7968, 155), (6141, 1386, 2404), (7532, 784, 2532), (8558, 270, 2730)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products_of_whole_numbers_are_exact(xm, m, n, k):
    torch = torch_cuda()
    for b_block_rows, a_block_rows, name in ((128, 1, "f32"), (1, 1, "bf16"), (1, 128, "f32")):
        dtype, _ = _type(torch, name)
        a, sa = _whole(torch, m, k, a_block_rows, m + n)
        b, sb = _whole(torch, n, k, b_block_rows, n + k)
        want = _values(torch, a, sa, a_block_rows) @ _values(torch, b, sb, b_block_rows).t()
        c, buf = _matrix(torch, m, n, dtype, pad=3, offset=1)
        xm.xp_matmul8(a, sa, b, sb, c, a_block_rows, b_block_rows)
        assert torch.equal(c, want.to(dtype)), (m, n, k, name, int((c != want.to(dtype)).sum()))
        assert torch.isnan(buf[1:1 + m * (n + 3)].view(m, n + 3)[:, n:]).all()    # nothing between the rows
        if name == "f32":
            xm.xp_matmul8(a, sa, b, sb, c, a_block_rows, b_block_rows, accumulate=True)
            assert torch.equal(c, (2 * want).float())


@pytest.mark.parametrize("m", [*range(1, 20), 31, 32, 33, 47, 63, 65, 95, 97, 127, 161, 193, 223, 225, 241, 257, 290])
def test_every_number_of_rows(xm, m):
    torch = torch_cuda()
    for n, k in ((260, 1536), (3000, 260)):
        a, sa = _whole(torch, m, k, 1, m)
        b, sb = _whole(torch, n, k, 128, 99)
        c = torch.full((m, n), float("nan"), device="cuda")
        xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128)
        assert torch.equal(c, (_values(torch, a, sa, 1) @ _values(torch, b, sb, 128).t()).float()), (m, n, k)


@pytest.mark.parametrize("m,n,k", [(1, 513, 4096), (64, 4096, 4096), (300, 1000, 1000), (1000, 3000, 12800), (512, 4096, 16001)])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_products_of_numbers(xm, m, n, k, name):
    # Products are exact.  The tensor core adds 32 of them to the sum at a time and may round towards zero after aligning
    # them, two units of 2^-23 of the magnitudes' sum at most each time, 4096 columns in a row; the parts are added in fp32.
    torch = torch_cuda()
    dtype, uo = _type(torch, name)
    rng = np.random.default_rng(k)
    x = rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)))
    w = rng.standard_normal((n, k)) * k ** -0.5
    a, sa, b, sb = _bytes(torch, m, k), _bytes(torch, m, _ceil(k, 128), 4), _bytes(torch, n, k), _bytes(torch, _ceil(n, 128), _ceil(k, 128), 4)
    xm.xp_block8_encode(torch.from_numpy(x).float().cuda(), a, sa)
    xm.xp_block8_encode(torch.from_numpy(w).float().cuda(), b, sb, block_rows=128)
    av, bv = _values(torch, a, sa, 1), _values(torch, b, sb, 128)
    want, size = av @ bv.t(), av.abs() @ bv.abs().t()
    bound = (min(k, 4096) / 32 + 2) * 2.0 ** -22 * size + (k / 4096 + 9) * U * size
    bound = bound + uo * (want.abs() + bound)
    c = torch.empty(m, n, dtype=dtype, device="cuda")
    xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128)
    assert ((c.double() - want).abs() <= bound).all(), float(((c.double() - want).abs() / bound).max())
    again = torch.empty_like(c)
    xm.xp_matmul8(a, sa, b, sb, again, b_block_rows=128)
    assert torch.equal(c, again)
    if name == "f32":   # on the average far below: as near as a plain fp32 sum of as many terms may be
        assert float((c.double() - want).norm() / want.norm()) < 2e-6


def test_scales_of_every_size(xm):
    # each row and column with a scale of its own: c[i, j] = k 2^(i - 127) 2^(j - 127), exact where fp32 has it as a normal number
    torch = torch_cuda()
    k = 128
    one = torch.full((255, k), 0x38, dtype=torch.uint8, device="cuda")
    scales = _bytes(torch, 255, 1, 4)
    scales.copy_(torch.arange(255, dtype=torch.uint8)[:, None])
    c = torch.empty(255, 255, device="cuda")
    xm.xp_matmul8(one, scales, one, scales, c)
    e = torch.arange(255)[:, None] + torch.arange(255)[None, :] - 254 + 7
    normal = (e >= -126) & (e <= 127)
    got = c.double().cpu()
    assert torch.equal(got[normal], torch.ldexp(torch.ones(1, dtype=torch.float64), e)[normal])
    assert (got[e < -149] == 0).all() and torch.isinf(got[e > 127]).all()


@pytest.mark.parametrize("m,n,k", [(3, 200, 640), (1, 4096, 2048), (600, 3000, 384)])
def test_a_block_that_is_not_a_number(xm, m, n, k):
    torch = torch_cuda()
    a, sa = _whole(torch, m, k, 1, 1)
    b, sb = _whole(torch, n, k, 128, 2)
    want = (_values(torch, a, sa, 1) @ _values(torch, b, sb, 128).t()).float()
    c = torch.empty(m, n, device="cuda")
    if m > 1:
        sa[1, -1] = 255
        xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128)
        assert torch.isnan(c[1]).all() and torch.equal(c[torch.arange(m) != 1], want[torch.arange(m) != 1])
        sa[1, -1] = 127
        want[1] = (_values(torch, a, sa, 1)[1] @ _values(torch, b, sb, 128).t()).float()
    sb[1, 0] = 255
    xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128)
    cols = torch.arange(n) // 128 == 1
    assert torch.isnan(c[:, cols]).all() and torch.equal(c[:, ~cols], want[:, ~cols])
    a[0, 5] = 0x7F     # a code
    sb[1, 0] = 127
    xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128)
    assert torch.isnan(c[0]).all() and (m == 1 or not torch.isnan(c[1:]).any())


def test_empty_products(xm):
    torch = torch_cuda()
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    c, _ = _matrix(torch, 5, 7, torch.float32, pad=2, fill=3.0)
    xm.xp_matmul8(z(5, 0), z(5, 0), z(7, 0), z(7, 0), c, accumulate=True)
    assert (c == 3).all()
    xm.xp_matmul8(z(5, 0), z(5, 0), z(7, 0), z(7, 0), c)
    assert (c == 0).all() and (c._base[35 + 10:] == 3).all()
    xm.xp_matmul8(z(0, 64), z(0, 1), z(7, 64), z(7, 1), torch.empty(0, 7, device="cuda"))
    xm.xp_matmul8(z(5, 64), z(5, 1), z(0, 64), z(0, 1), torch.empty(5, 0, device="cuda"))
    torch.cuda.synchronize()


def test_offsets_past_32_bits(xm):
    torch = torch_cuda()
    # c's rows 2^22 elements apart; a's codes 65536 bytes apart
    m, n, k = 1100, 130, 128
    a, sa = _whole(torch, m, k, 1, 1)
    b, sb = _whole(torch, n, k, 1, 2)
    want = (_values(torch, a, sa, 1) @ _values(torch, b, sb, 1).t()).bfloat16()
    wide = torch.zeros(m, 1 << 22, dtype=torch.bfloat16, device="cuda")
    xm.xp_matmul8(a, sa, b, sb, wide[:, -n:])
    assert torch.equal(wide[:, -n:], want) and not wide[:, : -n].any()
    del wide
    m = 70000
    wide = torch.zeros(m, 65536, dtype=torch.uint8, device="cuda")
    a, sa = _whole(torch, m, k, 1, 3)
    wide[:, 4096:4096 + k] = a
    c = torch.empty(m, n, device="cuda")
    xm.xp_matmul8(wide[:, 4096:4096 + k], sa, b, sb, c)
    av, bv = _values(torch, a, sa, 1), _values(torch, b, sb, 1)
    assert torch.equal(c, (av @ bv.t()).float())


# ---------------------------------------------------------------- root-mean-square norm

ROWS = [(1, 1), (3, 2), (5, 7), (2, 31), (9, 33), (4, 128), (17, 129), (33, 255), (6, 256), (130, 768), (5, 1000), (64, 1031), (11, 2048), (3, 4095), (2, 4096), (2, 8192),
        (3, 8200), (2, 16384), (2, 16385), (1, 20000), (2, 70001), (1, 1 << 20), (700, 520)]


def _norm_inputs(torch, rows, cols, dtype, wdtype, pad=0, offset=0, seed=0):
    rng = np.random.default_rng(seed + 1000 * rows + cols)
    make = lambda scale: _matrix(torch, rows, cols, dtype, pad, offset, values=rng.standard_normal((rows, cols)) * scale)[0]  # noqa: E731
    gamma = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).to(wdtype).cuda()
    return make(rng.uniform(0.2, 3, (rows, 1))), make(1.0), make(0.1), make(0.05), gamma


def _check_norm_forward(torch, xm, rows, cols, name, wname, pad=0, offset=0, residual=True, affine=True, eps=1e-5, out8=True):
    dtype, uo = _type(torch, name)
    x, r, _, _, gamma = _norm_inputs(torch, rows, cols, dtype, _type(torch, wname)[0], pad, offset)
    gamma = gamma if affine else None
    added = _matrix(torch, rows, cols, dtype, pad, offset)[0] if residual else None
    y, buf = _matrix(torch, rows, cols, dtype, pad, offset)
    rstd = torch.empty(rows, device="cuda")
    y8, s8 = (_bytes(torch, rows, cols, 16 if pad % 8 == 0 else 1), _bytes(torch, rows, _ceil(cols, 128), 1)) if out8 else (None, None)
    xm.xp_rmsnorm_forward(x, gamma, y, r if residual else None, added, rstd, y8, s8, eps)
    h = _f64(x)
    if residual:
        h = _f64((x.float() + r.float()).to(dtype))
        assert np.array_equal(_f64(added), h)
    want, want_rstd = model.rmsnorm_forward(h, None if gamma is None else _f64(gamma), float(np.float32(eps)))
    # a thread's chain of squares, 10 shuffle and CTA levels (32 warps one after another)
    er = 0.5 * (32 + cols / 1024 + 40) * U + 4 * U
    assert (np.abs(_f64(rstd) - want_rstd) <= er * want_rstd).all()
    ey = (er + 3 * U) * np.abs(want)
    assert (np.abs(_f64(y) - want) <= ey + uo * (np.abs(want) + ey)).all()
    if pad:
        assert torch.isnan(buf[offset:offset + rows * (cols + pad)].view(rows, -1)[:, cols:]).all()
    if out8:
        codes, scales = y8.cpu().numpy(), s8.cpu().numpy()
        padded = np.pad(want, ((0, 0), (0, -cols % 128))).reshape(rows, -1, 128)
        top, off = np.abs(padded).max(2), (er + 3 * U)
        assert ((scales == model.scale_of(top * (1 - off))) | (scales == model.scale_of(top * (1 + off)))).all()
        power = np.repeat(2.0 ** (scales.astype(int) - 127), 128, 1)[:, :cols]
        with np.errstate(divide="ignore"):
            half = np.maximum(2.0 ** np.floor(np.log2(np.abs(want) * (1 + off))), power * 2.0 ** -6) / 16
        assert (np.abs(model.decode(codes, scales) - want) <= half + ey).all()
        assert (y8._base[:, cols:] == 0x7F).all() and (s8._base[:, s8.shape[1]:] == 0x7F).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_norm_forward(xm, rows, cols, name):
    torch = torch_cuda()
    _check_norm_forward(torch, xm, rows, cols, name, "f32")
    _check_norm_forward(torch, xm, rows, cols, name, "bf16", residual=False, affine=cols % 2 == 0)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (6, 2), (3, 5), (0, 8)])
@pytest.mark.parametrize("rows,cols", [(5, 40), (7, 513), (3, 1024), (2, 9001), (2, 20000)])
def test_norm_strides_and_alignment(xm, rows, cols, pad, offset):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        _check_norm_forward(torch, xm, rows, cols, name, "f32", pad, offset)
        _check_norm_backward(torch, xm, rows, cols, name, "bf16", pad, offset)


@pytest.mark.parametrize("cols", [256, 1000, 20000])
def test_norm_forward_in_place_and_parts(xm, cols):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        dtype, _ = _type(torch, name)
        x, r, _, _, gamma = _norm_inputs(torch, 9, cols, dtype, torch.float32)
        added, y = torch.empty(9, cols, dtype=dtype, device="cuda"), torch.empty(9, cols, dtype=dtype, device="cuda")
        xm.xp_rmsnorm_forward(x, gamma, y, r, added)
        for into in ("x", "residual"):       # added into one input, y into the other
            a, b = x.clone(), r.clone()
            xm.xp_rmsnorm_forward(a, gamma, b if into == "x" else a, b, a if into == "x" else b)
            assert torch.equal(a if into == "x" else b, added) and torch.equal(b if into == "x" else a, y)
        a = x.clone()
        alone = torch.empty_like(a)
        xm.xp_rmsnorm_forward(a, gamma, alone)
        xm.xp_rmsnorm_forward(a, gamma, a)
        assert torch.equal(a, alone)
        # the 8-bit output alone is that with y
        y8, s8, z8, t8 = _bytes(torch, 9, cols), _bytes(torch, 9, _ceil(cols, 128), 4), _bytes(torch, 9, cols), _bytes(torch, 9, _ceil(cols, 128), 4)
        xm.xp_rmsnorm_forward(x, gamma, y, r, added, None, y8, s8)
        xm.xp_rmsnorm_forward(x, gamma, None, r, added, None, z8, t8)
        assert torch.equal(y8, z8) and torch.equal(s8, t8)


def test_norm_of_zeros_and_of_what_is_not_finite(xm):
    torch = torch_cuda()
    x = torch.zeros(4, 300, device="cuda")
    x[1, 7], x[2, 299], x[3] = float("inf"), float("nan"), 1e-30
    y, rstd = torch.empty_like(x), torch.empty(4, device="cuda")
    y8, s8 = _bytes(torch, 4, 300), _bytes(torch, 4, 3, 4)
    xm.xp_rmsnorm_forward(x, None, y, None, None, rstd, y8, s8, eps=0.0)
    assert torch.isinf(rstd[0]) and torch.isnan(y[0]).all() and (s8[0] == 255).all() and (y8[0] == 0x7F).all()   # 0 / 0
    assert torch.isnan(y[1, 7]) and (y[1, :7] == 0).all() and s8[1].tolist() == [255, 0, 0]
    assert torch.isnan(y[2]).all() and (s8[2] == 255).all()
    xm.xp_rmsnorm_forward(x, None, y, None, None, rstd, y8, s8)
    assert (y[0] == 0).all() and (s8[0] == 0).all() and (y8[0] == 0).all() and torch.allclose(y[3], torch.full_like(y[3], 1e-30 * 1e-5 ** -0.5))


def _check_norm_backward(torch, xm, rows, cols, name, wname, pad=0, offset=0, dadded=True, affine=True, dgamma=True, accumulate=False, in_place=None):
    dtype, uo = _type(torch, name)
    h, _, dy, d, gamma = _norm_inputs(torch, rows, cols, dtype, _type(torch, wname)[0], pad, offset)
    gamma = gamma if affine else None
    rstd = torch.from_numpy(model.rmsnorm_forward(_f64(h))[1]).float().cuda()
    h64, dy64, d64, r64, g64 = _f64(h), _f64(dy), _f64(d) if dadded else None, _f64(rstd), None if gamma is None else _f64(gamma)
    dx, buf = _matrix(torch, rows, cols, dtype, pad, offset)
    dx = {None: dx, "dy": dy, "dadded": d}[in_place]
    start = torch.full((cols,), 0.25 if accumulate else float("nan"), device="cuda")
    dg = start.clone() if dgamma else None
    work = torch.full((max(16, xm.xp_rmsnorm_workspace(rows, cols)),), 0xFF, dtype=torch.uint8, device="cuda")
    xm.xp_rmsnorm_backward(dy, h, gamma, rstd, dx, dg, work, d if dadded else None, accumulate)
    want, want_g = model.rmsnorm_backward(dy64, h64, g64, r64, d64)
    a, xhat = np.abs(dy64 if g64 is None else dy64 * g64), np.abs(h64 * r64[:, None])
    along = (a * xhat).mean(1, keepdims=True)
    # a and xhat once rounded each, their sum over a row, the products and differences of dx
    chain = (32 + cols / 1024 + 45) * U
    err = r64[:, None] * (xhat * along * (chain + 8 * U) + 6 * U * (a + xhat * along)) + 2 * U * (0 if d64 is None else np.abs(d64)) + 2 * U * np.abs(want)
    assert (np.abs(_f64(dx) - want) <= err + uo * (np.abs(want) + err)).all(), (rows, cols, name)
    if pad and in_place is None:
        assert torch.isnan(buf[offset:offset + rows * (cols + pad)].view(rows, -1)[:, cols:]).all()
    if dgamma:
        want_g = want_g + (0.25 if accumulate else 0)
        terms = np.abs(dy64) * xhat
        # one CTA's rows one after another (152 CTAs of one row at a time at least), its groups, then 32 chains of parts and 6 levels
        bound = (rows / 100 + 8 + 64 + 8) * U * terms.sum(0) + 3 * U * (terms.sum(0) + np.abs(want_g))
        assert (np.abs(_f64(dg) - want_g) <= bound).all(), (rows, cols, name)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_norm_backward(xm, rows, cols, name):
    torch = torch_cuda()
    _check_norm_backward(torch, xm, rows, cols, name, "f32")
    _check_norm_backward(torch, xm, rows, cols, name, "bf16", dadded=False, affine=cols % 2 == 0, accumulate=True)
    _check_norm_backward(torch, xm, rows, cols, name, "f32", dgamma=False, in_place="dy")
    _check_norm_backward(torch, xm, rows, cols, name, "f32", in_place="dadded")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(5001, 96), (4999, 95), (2500, 1032), (1201, 4104), (601, 5120), (400, 6200), (330, 8200), (310, 8191), (700, 3001),
                                       (620, 4097), (2400, 515), (3100, 33), (640, 6145), (330, 12000), (200, 16384), (160, 16392)])
def test_norm_backward_many_rows(xm, rows, cols, name):
    torch = torch_cuda()
    _check_norm_backward(torch, xm, rows, cols, name, "f32")


@pytest.mark.parametrize("rows,cols", [(1, 64), (700, 513), (3000, 128), (1000, 5120), (40, 8200)])
def test_norm_weight_gradient_of_whole_numbers_is_exact(xm, rows, cols):
    # rstd 1, small whole numbers: every order of additions gives the same, and a row left out or taken twice shows
    torch = torch_cuda()
    gen = torch.Generator("cuda").manual_seed(rows)
    h, dy = (torch.randint(-4, 5, (rows, cols), generator=gen, device="cuda").float() for _ in range(2))
    for dtype in (torch.float32, torch.bfloat16):
        dg = torch.empty(cols, device="cuda")
        work = torch.empty(xm.xp_rmsnorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        xm.xp_rmsnorm_backward(dy.to(dtype), h.to(dtype), None, torch.ones(rows, device="cuda"), torch.empty(rows, cols, dtype=dtype, device="cuda"), dg, work)
        assert torch.equal(dg, (dy * h).sum(0))


def test_norm_without_rows(xm):
    torch = torch_cuda()
    e, dg = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    assert xm.xp_rmsnorm_workspace(0, 40) == 0
    xm.xp_rmsnorm_forward(e, None, e)
    xm.xp_rmsnorm_backward(e, e, None, torch.empty(0, device="cuda"), e, dg, accumulate=True)
    assert (dg == 1).all()
    xm.xp_rmsnorm_backward(e, e, None, torch.empty(0, device="cuda"), e, dg)
    assert (dg == 0).all()


def test_norm_offsets_past_32_bits(xm):
    torch = torch_cuda()
    rows, cols = 70, 512
    wide = torch.zeros(rows, 1 << 26, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    wide[:, :cols] = x
    y, want = torch.empty_like(x), torch.empty_like(x)
    xm.xp_rmsnorm_forward(wide[:, :cols], None, wide[:, cols:2 * cols])
    xm.xp_rmsnorm_forward(x, None, want)
    assert torch.equal(wide[:, cols:2 * cols], want) and not wide[:, 2 * cols:].any()
    xm.xp_rmsnorm_backward(wide[:, :cols], wide[:, cols:2 * cols], None, torch.ones(rows, device="cuda"), wide[:, -cols:])
    xm.xp_rmsnorm_backward(x, want, None, torch.ones(rows, device="cuda"), y)
    assert torch.equal(wide[:, -cols:], y)


# ---------------------------------------------------------------- distillation

VOCABS = [(1, 1, 1), (2, 3, 2), (3, 31, 5), (5, 64, 1), (7, 127, 40), (4, 1000, 8), (6, 1031, 64), (3, 4096, 100), (2, 50257, 50), (300, 2049, 16), (1, 160001, 1024), (2, 600, 1024)]


def _distill_inputs(torch, rows, vocab, top, dtype, pad=0, offset=0, spread=2.5):
    rng = np.random.default_rng(vocab + rows)
    z, _ = _matrix(torch, rows, vocab, dtype, pad, offset, values=rng.standard_normal((rows, vocab)) * spread)
    ids = rng.integers(0, vocab, (rows, top))                      # the same id more than once
    ids[rng.random((rows, top)) < 0.1] = -1
    ids[rng.random((rows, top)) < 0.05] = vocab
    t = rng.standard_normal((rows, top)) * 2
    t[rng.random((rows, top)) < 0.05] = -np.inf
    if rows > 2:
        ids[1] = -1
    ids[0, 0], t[0, 0] = vocab - 1, 1.0
    return z, torch.from_numpy(ids).int().cuda(), torch.from_numpy(t).float().cuda(), rng


def _check_distill(torch, xm, rows, vocab, top, name, temperature, pad=0, offset=0, in_place=False, spread=2.5):
    dtype, uo = _type(torch, name)
    z, ids, t, rng = _distill_inputs(torch, rows, vocab, top, dtype, pad, offset, spread)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    xm.xp_distill_forward(z, ids, t, loss, lse, temperature)
    z64, i64, t64, T = _f64(z), ids.cpu().numpy(), _f64(t), float(np.float32(temperature))
    want, want_lse = model.distill_forward(z64, i64, t64, T)
    p, there = model.teacher(i64, t64, vocab, T)
    # 1/T, times log2 e, is off by 3 U, the same for all; an exponent is rounded once; a power; a thread's chain and 30 levels
    big = np.abs(z64).max(1) / T
    e_sum = (vocab / 256 + 60) * U + POW + 4 * U * big
    e_lse = e_sum + 6 * U * (big + np.abs(want_lse)) + 4 * U
    assert (np.abs(_f64(lse) - want_lse) <= np.where(there.any(1), e_lse, 0)).all()
    u = np.where(there, t64 / T, 0)
    width = (np.abs(u).max(1) + 1)[:, None]
    e_p = (2 * POW + (top / 32 + 12) * U + 12 * U * width) * p                                     # of an entry's share
    term = np.abs(np.where(p > 0, np.log(np.where(p > 0, p, 1)), 0)) + np.abs(np.take_along_axis(z64, np.clip(i64, 0, vocab - 1), 1) / T - want_lse[:, None])
    e_term = e_lse[:, None] + 8 * U * (width + big[:, None] + term) + POW + (top / 32 + 12) * U
    e_loss = T * T * ((e_p * term + p * e_term).sum(1) + (top / 32 + 12) * U * (p * term).sum(1)) + 4 * U * np.abs(want)
    assert (np.abs(_f64(loss) - want) <= np.where(there.any(1), e_loss, 0)).all(), float((np.abs(_f64(loss) - want) / e_loss).max())

    given = torch.from_numpy(want_lse).float().cuda()
    dloss = torch.from_numpy(rng.uniform(-1, 2, rows)).float().cuda()
    out, buf = _matrix(torch, rows, vocab, dtype, pad, offset)
    out = z if in_place else out
    xm.xp_distill_backward(z, ids, t, given, dloss, out, temperature)
    d64 = model.distill_backward(z64, i64, t64, _f64(given), _f64(dloss), T)
    g = np.abs(_f64(dloss) * T)[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        q = np.where(there.any(1)[:, None], np.exp(np.minimum(z64 / T - _f64(given)[:, None], 100)), 0)
    shares, e_shares = np.zeros_like(z64), np.zeros_like(z64)
    for i in range(rows):
        np.add.at(shares[i], i64[i, there[i]], p[i, there[i]])
        np.add.at(e_shares[i], i64[i, there[i]], e_p[i, there[i]])
    err = g * (q * (POW + 6 * U * (np.abs(z64) / T + np.abs(want_lse)[:, None] + 1)) + e_shares + (top + 4) * U * shares) + 4 * U * np.abs(d64)
    # a power below 2^-126 is 0, and g times that is what is missing then: g 2^-126 at most; rounding below 2^-126 is off by less than that
    assert (np.abs(_f64(out) - d64) <= err + uo * (np.abs(d64) + err) + (1 + g) * 2.0 ** -126).all(), (rows, vocab, top, name)
    if pad and not in_place:
        assert torch.isnan(buf[offset:offset + rows * (vocab + pad)].view(rows, -1)[:, vocab:]).all()


@pytest.mark.parametrize("temperature", [1.0, 3.0, 0.5])
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", VOCABS)
def test_distill(xm, rows, vocab, top, name, temperature):
    _check_distill(torch_cuda(), xm, rows, vocab, top, name, temperature)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (6, 2), (3, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_distill_strides_alignment_and_in_place(xm, pad, offset, in_place):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        _check_distill(torch, xm, 5, 3000, 20, name, 2.0, pad, offset, in_place)
        _check_distill(torch, xm, 200, 777, 9, name, 1.0, pad, offset, in_place)


@pytest.mark.parametrize("vocab,top,pad,offset", [(1, 1, 0, 0), (40, 3, 1, 1), (512, 20, 0, 0), (1000, 64, 3, 5), (1024, 7, 0, 0)])
def test_distill_many_short_rows(xm, vocab, top, pad, offset):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        _check_distill(torch, xm, 5003, vocab, top, name, 1.0, pad, offset, pad > 0)


def test_distill_large_logits(xm):
    torch = torch_cuda()
    for spread in (30.0, 300.0):
        _check_distill(torch, xm, 4, 2000, 30, "f32", 1.0, spread=spread)


def test_distill_into_rows_of_another_phase(xm):
    torch = torch_cuda()
    z, ids, t, _ = _distill_inputs(torch, 4, 1001, 6, torch.bfloat16)
    loss, lse, d = (torch.empty(4, device="cuda") for _ in range(3))
    d.fill_(0.5)
    xm.xp_distill_forward(z, ids, t, loss, lse)
    want, other = torch.empty_like(z), _matrix(torch, 4, 1001, torch.bfloat16, 3, 1)[0]
    xm.xp_distill_backward(z, ids, t, lse, d, want)
    xm.xp_distill_backward(z, ids, t, lse, d, other)
    assert torch.equal(want, other)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_distill_masks_and_what_is_not_finite(xm, name):
    torch = torch_cuda()
    inf, nan = float("inf"), float("nan")
    dtype, _ = _type(torch, name)
    z = torch.zeros(8, 300, dtype=dtype, device="cuda")
    ids = torch.tensor([[3, 5]] * 8, dtype=torch.int32, device="cuda")
    t = torch.zeros(8, 2, device="cuda")
    z[0, 100:] = -inf                      # a masked vocabulary
    z[1, 5] = -inf                         # the teacher wants what is masked
    z[2] = -inf                            # nothing left
    z[3, 9] = nan
    z[4, 9] = inf
    z[5], ids[5] = nan, -1                 # a row without entries: its logits do not matter
    t[6] = -inf                            # nor here
    t[7, 1] = nan
    loss, lse, d = torch.empty(8, device="cuda"), torch.empty(8, device="cuda"), torch.ones(8, device="cuda")
    xm.xp_distill_forward(z, ids, t, loss, lse)
    assert torch.allclose(lse[0], torch.tensor(100.0, device="cuda").log()) and torch.isfinite(loss[0])
    assert loss[1] == inf and torch.isfinite(lse[1])
    assert torch.isnan(loss[[2, 3, 4, 7]]).all() and loss[5] == 0 == lse[5] and loss[6] == 0 == lse[6]
    g = torch.empty_like(z)
    xm.xp_distill_backward(z, ids, t, lse, d, g)
    assert (g[0, 100:] == 0).all() and torch.isfinite(g[0]).all() and g[1, 5] == -0.5 and torch.isfinite(g[1]).all()
    assert torch.isnan(g[3]).all() and (g[5] == 0).all() and (g[6] == 0).all() and torch.isnan(g[7, [3, 5]]).all()
    # a mask of the type's lowest value
    z[0, 100:] = torch.finfo(dtype).min
    xm.xp_distill_forward(z[:1], ids[:1], t[:1], loss[:1], lse[:1])
    assert torch.allclose(lse[0], torch.tensor(100.0, device="cuda").log())
    none = torch.empty(8, 0, dtype=torch.int32, device="cuda")
    xm.xp_distill_forward(z, none, none.float(), loss, lse)
    xm.xp_distill_backward(z, none, none.float(), lse, d, g)
    assert (loss == 0).all() and (g == 0).all()
    xm.xp_distill_forward(z[:0], ids[:0], t[:0], loss[:0], lse[:0])


def test_distill_offsets_past_32_bits(xm):
    torch = torch_cuda()
    rows, vocab = 70, 1000
    wide = torch.zeros(rows, 1 << 26, dtype=torch.bfloat16, device="cuda")
    z, ids, t, _ = _distill_inputs(torch, rows, vocab, 4, torch.bfloat16)
    wide[:, 8:8 + vocab] = z
    loss, lse, other, d = (torch.ones(rows, device="cuda") for _ in range(4))
    xm.xp_distill_forward(z, ids, t, loss, lse)
    xm.xp_distill_forward(wide[:, 8:8 + vocab], ids, t, other)
    assert torch.equal(loss, other)
    g = torch.empty_like(z)
    xm.xp_distill_backward(z, ids, t, lse, d, g)
    xm.xp_distill_backward(wide[:, 8:8 + vocab], ids, t, lse, d, wide[:, -vocab:])
    assert torch.equal(wide[:, -vocab:], g)


# ---------------------------------------------------------------- together

class Layer:
    """A last layer in 8 bits: norm of x + residual, a product with a weight, the loss; and back.  Every buffer is its own."""

    def __init__(self, torch, xm, rows, cols, vocab, top, seed):
        self.torch, self.xm, self.T = torch, xm, 2.0
        gen = torch.Generator("cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        b = lambda *s: _bytes(torch, *s)  # noqa: E731
        e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.x, self.r = n(rows, cols).to(bf), n(rows, cols).to(bf)
        self.gamma, self.w = 1 + 0.1 * n(cols), n(vocab, cols) * 2 * cols ** -0.5
        self.ids = torch.randint(-1, vocab, (rows, top), generator=gen, device="cuda", dtype=torch.int32)
        self.t, self.dloss = n(rows, top), torch.full((rows,), 1.0 / rows, device="cuda")
        blocks = lambda k: _ceil(k, 128)  # noqa: E731
        self.w8, self.sw, self.w8t, self.swt = b(vocab, cols), b(blocks(vocab), blocks(cols)), b(cols, vocab), b(blocks(cols), blocks(vocab))
        self.h, self.y, self.rstd, self.y8, self.sy = e(rows, cols, dtype=bf), e(rows, cols, dtype=bf), e(rows), b(rows, cols), b(rows, blocks(cols))
        self.y8t, self.syt = b(cols, rows), b(cols, blocks(rows))
        self.z, self.loss, self.lse, self.dz = e(rows, vocab), e(rows), e(rows), e(rows, vocab)
        self.dz8, self.sdz, self.dz8t, self.sdzt = b(rows, vocab), b(rows, blocks(vocab)), b(vocab, rows), b(vocab, blocks(rows))
        self.dy, self.dw, self.dx, self.dgamma = e(rows, cols, dtype=bf), torch.zeros(vocab, cols, device="cuda"), e(rows, cols, dtype=bf), e(cols)
        self.work = e(max(16, xm.xp_rmsnorm_workspace(rows, cols)), dtype=torch.uint8)

    def step(self, stream=None):
        xm = self.xm
        xm.xp_block8_encode(self.w, self.w8, self.sw, self.w8t, self.swt, block_rows=128, stream=stream)
        xm.xp_rmsnorm_forward(self.x, self.gamma, self.y, self.r, self.h, self.rstd, self.y8, self.sy, stream=stream)
        xm.xp_matmul8(self.y8, self.sy, self.w8, self.sw, self.z, b_block_rows=128, stream=stream)
        xm.xp_distill_forward(self.z, self.ids, self.t, self.loss, self.lse, self.T, stream=stream)
        xm.xp_distill_backward(self.z, self.ids, self.t, self.lse, self.dloss, self.dz, self.T, stream=stream)
        xm.xp_block8_encode(self.dz, self.dz8, self.sdz, self.dz8t, self.sdzt, stream=stream)
        xm.xp_block8_encode(self.y, codes_t=self.y8t, scales_t=self.syt, stream=stream)
        xm.xp_matmul8(self.dz8, self.sdz, self.w8t, self.swt, self.dy, b_block_rows=128, stream=stream)
        xm.xp_matmul8(self.dz8t, self.sdzt, self.y8t, self.syt, self.dw, accumulate=True, stream=stream)
        xm.xp_rmsnorm_backward(self.dy, self.h, self.gamma, self.rstd, self.dx, self.dgamma, self.work, stream=stream)

    def outputs(self):
        return [getattr(self, k).clone() for k in ("h", "y", "rstd", "y8", "sy", "z", "loss", "lse", "dz", "dz8", "dz8t", "dy", "dw", "dx", "dgamma")]


@pytest.mark.parametrize("rows,cols,vocab", [(5, 256, 1000), (70, 512, 3001), (600, 1032, 4096)])
def test_a_layers_step(xm, rows, cols, vocab):
    # without a pause between the calls; then every stage against its formula on what the stage before it gave
    torch = torch_cuda()
    s = Layer(torch, xm, rows, cols, vocab, 12, rows)
    s.step()
    n = lambda t: t.cpu().numpy()  # noqa: E731
    assert torch.equal(s.h, (s.x.float() + s.r.float()).bfloat16())
    for x, c, sc, block_rows in ((s.w, s.w8, s.sw, 128), (s.w.t(), s.w8t, s.swt, 128), (s.dz, s.dz8, s.sdz, 1), (s.dz.t(), s.dz8t, s.sdzt, 1), (s.y.t(), s.y8t, s.syt, 1)):
        codes, scales = model.encode(_f64(x), block_rows)
        assert np.array_equal(n(c), codes) and np.array_equal(n(sc), scales)
    for a, sa, b, sb, c, block_rows in ((s.y8, s.sy, s.w8, s.sw, s.z, 128), (s.dz8, s.sdz, s.w8t, s.swt, s.dy, 128), (s.dz8t, s.sdzt, s.y8t, s.syt, s.dw, 1)):
        want, size = model.product(n(a), n(sa), n(b), n(sb), 1, block_rows)
        k = a.shape[1]
        uo = 2.0 ** -8 if c.dtype == torch.bfloat16 else U
        assert (np.abs(_f64(c) - want) <= (k / 32 + 4) * 2.0 ** -22 * size + uo * np.abs(want) * 1.01).all()
    loss, lse = model.distill_forward(_f64(s.z), n(s.ids), _f64(s.t), s.T)
    assert np.allclose(_f64(s.loss), loss, rtol=1e-4, atol=1e-4) and np.allclose(_f64(s.lse), lse, rtol=1e-5)
    dx, dgamma = model.rmsnorm_backward(_f64(s.dy), _f64(s.h), _f64(s.gamma), _f64(s.rstd))
    scale = np.abs(dx).max()
    assert np.abs(_f64(s.dx) - dx).max() <= 2.0 ** -7 * scale and np.abs(_f64(s.dgamma) - dgamma).max() <= 1e-4 * np.abs(dgamma).max()


def test_a_steps_gradient_is_that_of_differences(xm):
    # dgamma along a direction against the loss at gamma +- step, both through 8 bits.  A product's operands are each off by
    # half a step of 2^-3, 2^-4 of themselves, and errors of opposite sign cancel: over 64 x 512 terms the directional
    # derivative keeps more than nine tenths.
    torch = torch_cuda()
    s = Layer(torch, xm, 64, 512, 1000, 12, 3)
    s.step()
    direction = s.dgamma / s.dgamma.norm()
    predicted, start = float((s.dgamma * direction).sum()), s.gamma.clone()
    values = []
    for sign in (1, -1):
        s.gamma = start + sign * 0.5 * direction
        s.step()
        values.append(float((s.loss * s.dloss).sum()))
    assert abs((values[0] - values[1]) / 1.0 / predicted - 1) < 0.1


def test_steps_in_graphs_and_on_streams(xm):
    # two layers at a time on two streams, each captured and replayed with other inputs, give what they give alone
    torch = torch_cuda()
    layers = [Layer(torch, xm, 130, 520, 1500, 9, 1), Layer(torch, xm, 33, 1024, 2049, 9, 2)]
    others = [Layer(torch, xm, 130, 520, 1500, 9, 3), Layer(torch, xm, 33, 1024, 2049, 9, 4)]
    want = []
    for s, o in zip(layers, others):
        o.step()
        want.append(o.outputs())
        s.step()
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in layers], []
    for s, st in zip(layers, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            s.step(st)
        graphs.append(g)
    for s, o in zip(layers, others):
        for k in ("x", "r", "gamma", "w", "ids", "t"):
            getattr(s, k).copy_(getattr(o, k))
    torch.cuda.synchronize()
    for _ in range(3):
        for s in layers:
            s.dw.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(layers, want):
            assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w))


def test_products_at_once_and_first_called_in_a_capture(xm):
    # clusters of two pairs, pairs, CTAs that share a tile: a process's first products are captured, and replayed at once
    code = """
import sys
sys.path.insert(0, %r)
import torch
from collective_transport_plane_gb300 import xp_model as xm
sizes, calls = [(801, 6595, 2148), (4186, 1320, 1666), (2000, 700, 2001), (1, 4096, 4096)], []
for i, (m, n, k) in enumerate(sizes):
    g = torch.Generator().manual_seed(i)
    pitch, kb = (k + 15) // 16 * 16, (k + 127) // 128
    codes = [(torch.randint(0, 2, (r, pitch), generator=g) * 0x38).to(torch.uint8).cuda()[:, :k] for r in (m, n)]      # 0 or 1
    scales = [torch.full((r, (kb + 3) // 4 * 4), 127, dtype=torch.uint8, device="cuda")[:, :kb] for r in (m, n)]
    want = (codes[0].double() / 0x38) @ (codes[1].double() / 0x38).t()
    calls.append((codes, scales, want.float(), torch.zeros(m, n, device="cuda")))
torch.cuda.synchronize()
graphs = []
for (a, b), (sa, sb), want, c in calls:
    graphs.append((torch.cuda.CUDAGraph(), torch.cuda.Stream()))
    with torch.cuda.graph(graphs[-1][0], stream=graphs[-1][1]):
        xm.xp_matmul8(a, sa, b, sb, c, stream=graphs[-1][1])
for _ in range(5):
    for *_, c in calls:
        c.fill_(-1)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for *_, want, c in calls)
assert xm.xp_matmul8_status() == 0
print("equal")
""" % ROOT
    torch_cuda()
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip().endswith("equal"), done.stderr[-2000:]


def test_calls_of_threads(xm):
    import threading
    torch = torch_cuda()
    layers = [Layer(torch, xm, 40 + 30 * i, 384, 1200, 7, i) for i in range(4)]
    for s in layers:
        s.step()
    torch.cuda.synchronize()
    want = [s.outputs() for s in layers]

    def work(s):
        st = torch.cuda.Stream()
        for _ in range(20):
            with torch.cuda.stream(st):
                s.dw.zero_()
            s.step(st)
        st.synchronize()

    threads = [threading.Thread(target=work, args=(s,)) for s in layers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for s, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w))


def test_tensors_of_the_host_are_refused(xm):
    torch = torch_cuda()
    x = torch.zeros(4, 256, device="cuda")
    with pytest.raises(ValueError):
        xm.xp_rmsnorm_forward(x, None, torch.zeros(4, 256))
    with pytest.raises(ValueError):
        xm.xp_rmsnorm_forward(torch.zeros(4, 256), None, torch.zeros(4, 256))

"""The training operators on the GPU against their formulas in 64 bits (oracle.train), within bounds that follow from
fp32 rounding.

u = 2^-24 is fp32's rounding error, uo that of the output's type.  A row's sums go through at most 16 terms per thread
and column block, 10 shuffle levels and 8 cluster ranks: SUM = 40 additions deep covers every path, so a sum of n terms
is off by at most 40 u times the sum of their magnitudes, and a mean by 42 u times the mean magnitude."""
import numpy as np
import pytest

from oracle import train
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 42 * U


@pytest.fixture(scope="module")
def xt():
    torch_cuda()
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_train as xt
    return xt


def _types(torch, name):
    """The type, and what rounding to it may be off relatively (bf16 keeps 8 bits: 2^-8; fp32's is counted in U)."""
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[name]
    return dtype, 0.0 if name == "f32" else torch.finfo(dtype).eps / 2


def _f64(t):
    return t.double().cpu().numpy()


def _matrix(torch, values, dtype, pad=0, offset=0):
    """A rows x cols view whose rows are pad elements further apart and whose first element is `offset` elements into
    its buffer; the elements between hold NaN."""
    rows, cols = values.shape
    buf = torch.full((offset + rows * (cols + pad) + 16,), float("nan"), dtype=dtype, device="cuda")
    m = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.from_numpy(values).to(dtype))
    return m


def _inputs(torch, rows, cols, dtype, wdtype, pad=0, offset=0, seed=0, shift=0.0):
    rng = np.random.default_rng(seed + 1000 * rows + cols)
    x = rng.standard_normal((rows, cols)) * rng.uniform(0.2, 3, (rows, 1)) + shift + rng.standard_normal((rows, 1))
    dy = rng.standard_normal((rows, cols)) * 0.1 + 0.02
    xm, dm = _matrix(torch, x, dtype, pad, offset), _matrix(torch, dy, dtype, pad, offset)
    gamma = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).to(wdtype).cuda()
    beta = torch.from_numpy(0.2 * rng.standard_normal(cols)).to(wdtype).cuda()
    return xm, dm, gamma, beta


def _forward_bounds(x, gamma, beta, eps, uo):
    """(y, mean, rstd, their bounds) from float64 arrays."""
    y, mean, rstd = train.layernorm_forward(x, gamma, beta, eps)
    em = SUM * np.abs(x).mean(1)
    d = np.abs(x - mean[:, None])
    var = (d ** 2).mean(1)
    er = 0.5 * ((SUM + 4 * U) * var + em ** 2 + 2 * U * np.abs(mean) * em) / (var + eps) + 4 * U    # relative
    xhat = d * rstd[:, None]
    exh = rstd[:, None] * (em[:, None] + U * (d + em[:, None])) + xhat * (er[:, None] + 3 * U)
    g = np.ones_like(y) if gamma is None else np.abs(gamma)[None, :] * np.ones_like(y)
    ey = g * exh + 3 * U * (xhat * g + np.abs(y))
    ey = ey + uo * (np.abs(y) + ey)
    return y, mean, rstd, ey, em + U * np.abs(mean), er * rstd * 1.01 + U * rstd


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 31), (9, 33), (17, 64), (4, 100), (33, 255), (6, 256), (7, 257), (130, 768), (5, 1000), (64, 1031),
          (11, 2048), (3, 4095), (2, 4104), (200, 513), (3, 8192), (2, 8193), (1, 16384), (2, 16390), (160, 4200), (1, 40001),
          (3, 65536), (1, 131072), (400, 9000)]


def _check_forward(torch, xt, rows, cols, name, wname, pad=0, offset=0, affine=True, shift=0.0, eps=1e-5):
    dtype, uo = _types(torch, name)
    wdtype, _ = _types(torch, wname)
    x, _, gamma, beta = _inputs(torch, rows, cols, dtype, wdtype, pad, offset, shift=shift)
    if not affine:
        gamma = beta = None
    y = _matrix(torch, np.zeros((rows, cols)), dtype, pad, offset)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    xt.xp_layernorm_forward(x, gamma, beta, y, mean, rstd, eps)
    want = _forward_bounds(_f64(x), None if gamma is None else _f64(gamma), None if beta is None else _f64(beta), float(np.float32(eps)), uo)
    for got, ref, bound in zip((y, mean, rstd), want[:3], want[3:]):
        off = np.abs(_f64(got) - ref)
        assert (off <= bound).all(), (rows, cols, float((off / bound).max()))
    if pad:   # nothing between the rows is written
        buf = y._base if y._base is not None else y
        assert torch.isnan(buf.flatten()[offset:offset + rows * (cols + pad)].view(rows, -1)[:, cols:]).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(xt, rows, cols, name):
    torch = torch_cuda()
    _check_forward(torch, xt, rows, cols, name, "f32")
    _check_forward(torch, xt, rows, cols, name, "bf16", affine=cols % 2 == 0)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (6, 2), (3, 5), (0, 4)])
@pytest.mark.parametrize("rows,cols", [(5, 40), (7, 513), (3, 1024), (2, 9001), (2, 20000)])
def test_forward_strides_and_alignment(xt, rows, cols, pad, offset):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        _check_forward(torch, xt, rows, cols, name, "f32", pad, offset)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(5001, 96), (4999, 95), (6000, 256), (700, 1100), (330, 1536), (330, 1537), (320, 9000), (160, 20000),
                                       (155, 32768), (160, 40032), (158, 40031), (155, 66001), (153, 70000)])
def test_forward_many_rows(xt, rows, cols, name):
    torch = torch_cuda()
    _check_forward(torch, xt, rows, cols, name, "f32")


@pytest.mark.parametrize("rows,cols", [(620, 2056), (611, 2401), (620, 2560), (700, 1704), (650, 1792), (609, 4104), (613, 5119), (610, 5120), (615, 7000),
                                       (608, 12001), (612, 16384), (607, 9000)])
def test_forward_threads_of_40_and_64(xt, rows, cols):
    torch = torch_cuda()
    for wname in ("f32", "bf16"):
        _check_forward(torch, xt, rows, cols, "bf16", wname)


@pytest.mark.parametrize("cols", [64, 1024, 1704, 2400, 4096, 12000, 20000])
def test_forward_weights_aligned_to_16_and_32_bytes(xt, cols):
    torch = torch_cuda()
    x, _, gamma, beta = _inputs(torch, 330, cols, torch.bfloat16, torch.float32)
    got = []
    for at in (0, 4, 8, 12):
        g, b = (torch.full((cols + 16,), float("nan"), device="cuda")[at:at + cols].copy_(w) for w in (gamma, beta))
        y = torch.zeros(330, cols, dtype=torch.bfloat16, device="cuda")
        xt.xp_layernorm_forward(x, g, b, y)
        got.append(y)
    assert torch.isfinite(got[0]).all() and all(torch.equal(got[0], y) for y in got[1:])


def test_forward_far_from_zero_and_large_eps(xt):
    torch = torch_cuda()
    _check_forward(torch, xt, 20, 1536, "f32", "f32", shift=30.0)
    _check_forward(torch, xt, 20, 300, "bf16", "f32", shift=-10.0, eps=0.5)


def _check_backward(torch, xt, rows, cols, name, wname, pad=0, offset=0, affine=True, accumulate=False):
    dtype, uo = _types(torch, name)
    wdtype, _ = _types(torch, wname)
    x, dy, gamma, _ = _inputs(torch, rows, cols, dtype, wdtype, pad, offset, seed=5)
    if not affine:
        gamma = None
    x64, dy64, g64 = _f64(x), _f64(dy), None if gamma is None else _f64(gamma)
    _, mean64, rstd64 = train.layernorm_forward(x64)
    mean, rstd = torch.from_numpy(mean64).float().cuda(), torch.from_numpy(rstd64).float().cuda()
    dx = _matrix(torch, np.zeros((rows, cols)), dtype, pad, offset)
    start = np.random.default_rng(1).standard_normal((2, cols)).astype(np.float32)
    dgamma, dbeta = torch.from_numpy(start[0].copy()).cuda(), torch.from_numpy(start[1].copy()).cuda()
    work = torch.empty(xt.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, work, accumulate)
    mean64, rstd64 = _f64(mean), _f64(rstd)
    want, wg, wb = train.layernorm_backward(dy64, x64, g64, mean64, rstd64)
    r = rstd64[:, None]
    xhat = (x64 - mean64[:, None]) * r
    exh = 3 * U * np.abs(xhat)
    a = np.abs(dy64 if g64 is None else dy64 * g64)
    m1, m2 = a.mean(1, keepdims=True), (a * np.abs(xhat)).mean(1, keepdims=True)
    c2 = np.abs(((dy64 if g64 is None else dy64 * g64) * xhat).mean(1, keepdims=True))
    bound = r * (4 * U * (a + m1 + np.abs(xhat) * c2) + SUM * m1 + np.abs(xhat) * (SUM + 6 * U) * m2 + exh * c2) + 2 * U * np.abs(want)
    bound = bound + uo * (np.abs(want) + bound)
    off = np.abs(_f64(dx) - want)
    assert (off <= bound).all(), (rows, cols, float((off / np.maximum(bound, 1e-300)).max()))
    # a column's sum: a thread's rows one after the other (no more than all of them), the groups of a CTA, the parts in
    # fp64, one rounding
    deep = (rows + 20) * U
    for got, ref, mags, first in ((dgamma, wg, np.abs(dy64 * xhat).sum(0), start[0]), (dbeta, wb, np.abs(dy64).sum(0), start[1])):
        ref = ref + first.astype(np.float64) if accumulate else ref
        assert (np.abs(_f64(got) - ref) <= (deep + 6 * U) * mags + 2 * U * np.abs(ref)).all()
    if pad:
        buf = dx._base if dx._base is not None else dx
        assert torch.isnan(buf.flatten()[offset:offset + rows * (cols + pad)].view(rows, -1)[:, cols:]).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(xt, rows, cols, name):
    torch = torch_cuda()
    _check_backward(torch, xt, rows, cols, name, "f32")
    _check_backward(torch, xt, rows, cols, name, "bf16", affine=cols % 2 == 0, accumulate=True)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (6, 2), (3, 5), (0, 4)])
@pytest.mark.parametrize("rows,cols", [(5, 40), (700, 130), (7, 513), (300, 1024), (2, 9001), (2, 20000)])
def test_backward_strides_and_alignment(xt, rows, cols, pad, offset):
    torch = torch_cuda()
    for name in ("f32", "bf16"):
        _check_backward(torch, xt, rows, cols, name, "f32", pad, offset)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(40, 1), (5000, 95), (37, 257), (300, 601), (40, 1031), (700, 1505), (330, 1793), (9, 4097), (3, 9001), (2, 40001)])
def test_each_tensor_has_its_own_alignment(xt, rows, cols, name):
    """Rows of odd lengths: where each matrix and the weights begin, and how far apart their rows are, changes no bit."""
    torch = torch_cuda()
    dtype, _ = _types(torch, name)
    rng = np.random.default_rng(rows + cols)
    x, dy = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    weights = [torch.from_numpy(rng.standard_normal(cols)).to(t) for t in (torch.float32, torch.bfloat16)]
    work = torch.empty(xt.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    first = {}
    for turn in range(9):
        place = rng.integers(0, 9, (4, 2)) if turn else np.zeros((4, 2), int)
        xm, dm = _matrix(torch, x, dtype, *map(int, place[0])), _matrix(torch, dy, dtype, *map(int, place[1]))
        y, dx = (_matrix(torch, np.zeros((rows, cols)), dtype, *map(int, place[k])) for k in (2, 3))
        for which, w in enumerate(weights):
            buf = torch.full((cols + 40,), float("nan"), dtype=w.dtype, device="cuda")
            gamma = buf[turn % 5:turn % 5 + cols]
            gamma.copy_(w)
            mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            xt.xp_layernorm_forward(xm, gamma, gamma, y, mean, rstd, 1e-5)
            xt.xp_layernorm_backward(dm, xm, gamma, mean, rstd, dx, dgamma, dbeta, work)
            got = [t.clone() for t in (y, mean, rstd, dx, dgamma, dbeta)]
            assert all(torch.isfinite(t).all() for t in got)
            for a, b in zip(got, first.setdefault(which, got)):
                assert torch.equal(a, b), (turn, which, place.tolist())
            for m, (pad, offset) in ((y, place[2]), (dx, place[3])):   # and nothing around the rows is written
                flat = m._base.flatten()
                assert torch.isnan(flat[:offset]).all() and torch.isnan(flat[offset + rows * (cols + pad):]).all()
                if pad:
                    assert torch.isnan(flat[offset:offset + rows * (cols + pad)].view(rows, -1)[:, cols:]).all()


@pytest.mark.parametrize("rows,cols", [(20000, 48), (5000, 1000), (1000, 6000)])
def test_backward_many_rows(xt, rows, cols):
    torch = torch_cuda()
    _check_backward(torch, xt, rows, cols, "bf16", "f32")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(30001, 96), (29999, 95), (9000, 257), (7001, 300), (3001, 2080), (2999, 2081), (1300, 5120),
                                       (1250, 8192), (620, 12000), (610, 12001), (170, 66000)])
def test_backward_more_rows(xt, rows, cols, name):
    torch = torch_cuda()
    _check_backward(torch, xt, rows, cols, name, "bf16", accumulate=cols % 2 == 1)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(9729, 8), (12003, 64), (10007, 120), (20001, 128), (305, 64), (611, 128), (4865, 16), (40000, 96)])
def test_rows_of_half_a_warp(xt, rows, cols, name):
    torch = torch_cuda()
    _check_forward(torch, xt, rows, cols, name, "f32")
    _check_forward(torch, xt, rows, cols, name, "bf16", pad=8)
    _check_backward(torch, xt, rows, cols, name, "f32", accumulate=True)
    _check_backward(torch, xt, rows, cols, name, "bf16", pad=8)


@pytest.mark.parametrize("rows", [306, 10007])
def test_half_warps_keep_bad_rows_apart(xt, rows):
    """Rows that hold an infinity or NaN leave every other row's bits as they are, the one of the warp's other half among them."""
    torch = torch_cuda()
    x, dy, gamma, beta = _inputs(torch, rows, 64, torch.bfloat16, torch.float32)
    bad = torch.arange(rows, device="cuda") % 3 == 1
    out = []
    for spoil in (False, True):
        if spoil:
            x[bad, 5] = float("inf")
            dy[bad, 7] = float("nan")
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        xt.xp_layernorm_forward(x, gamma, beta, y, mean, rstd, 1e-5)
        xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx)
        out.append([t[~bad].clone() for t in (y, mean, rstd, dx)])
        assert not spoil or (torch.isnan(y[bad]).any(1).all() and torch.isnan(dx[bad]).any(1).all())
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(*out))


@pytest.mark.parametrize("rows,cols", [(37, 200), (37, 1000), (5, 30000)])
def test_layernorm_in_place_repeatable_and_optional(xt, rows, cols):
    torch = torch_cuda()
    x, dy, gamma, beta = _inputs(torch, rows, cols, torch.bfloat16, torch.float32)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    xt.xp_layernorm_forward(x, gamma, beta, y, mean, rstd)
    z = x.clone()
    xt.xp_layernorm_forward(z, gamma, beta, z)
    assert torch.equal(y, z)
    outs = []
    work = torch.empty(xt.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        work.fill_(255)     # NaN in every word: what the last call left does not count
        dx, dg, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx, dg, db, work)
        outs.append((dx, dg, db))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    alone = torch.empty_like(x)
    xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, alone)
    d = dy.clone()
    xt.xp_layernorm_backward(d, x, gamma, mean, rstd, d)
    assert torch.equal(alone, outs[0][0]) and torch.equal(d, alone)


@pytest.mark.parametrize("cols", [60, 1000, 20000])
def test_layernorm_keeps_bad_rows_apart(xt, cols):
    torch = torch_cuda()
    x, dy, gamma, beta = _inputs(torch, 6, cols, torch.float32, torch.float32)
    x[1, 3], x[4, cols - 1] = float("nan"), float("inf")
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    xt.xp_layernorm_forward(x, gamma, beta, y, mean, rstd)
    fine = torch.tensor([0, 2, 3, 5])
    assert torch.isfinite(y[fine]).all() and torch.isnan(y[[1, 4]]).all()
    dx = torch.empty_like(x)
    xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx)
    assert torch.isfinite(dx[fine]).all() and torch.isnan(dx[[1, 4]]).all()


def test_layernorm_constant_rows(xt):
    # the variance is 0: y is beta, whatever the constant, as long as fp32 holds its mean exactly
    torch = torch_cuda()
    x = torch.tensor([0.0, 1.0, -4.0, 65536.0], device="cuda")[:, None].expand(4, 512).contiguous()
    beta = torch.randn(512, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(4, device="cuda")
    xt.xp_layernorm_forward(x, None, beta, y, None, rstd, 1e-4)
    assert torch.equal(y, beta.expand(4, 512))
    assert ((rstd - 100).abs() <= 100 * 8 * U).all()


def test_layernorm_no_rows_clears_the_sums(xt):
    torch = torch_cuda()
    x = torch.empty(0, 8, device="cuda")
    none = torch.empty(0, device="cuda")
    dg, db = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    xt.xp_layernorm_forward(x, None, None, x, none, none)
    xt.xp_layernorm_backward(x, x, None, none, none, x, dg, db, None, True)
    assert (dg == 1).all() and (db == 1).all()
    xt.xp_layernorm_backward(x, x, None, none, none, x, dg, db)
    assert (dg == 0).all() and (db == 0).all()


def test_layernorm_rows_far_apart(xt):
    # three rows 2^31 elements apart: offsets pass 32 bits
    torch = torch_cuda()
    rows, cols, stride = 3, 1000, 1 << 31
    buf = torch.empty(2 * stride + cols, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((rows, cols), (stride, 1))
    x, dy, gamma, beta = _inputs(torch, rows, cols, torch.bfloat16, torch.float32)
    far.copy_(x)
    out, mean, rstd = [], torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    work = torch.empty(xt.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    for a in (x, far):
        y, dx, dg, db = torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        xt.xp_layernorm_forward(a, gamma, beta, y, mean, rstd)
        xt.xp_layernorm_backward(dy, a, gamma, mean, rstd, dx, dg, db, work)
        out.append((y, dx, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    xt.xp_layernorm_forward(x, gamma, beta, far)
    assert torch.equal(far, out[0][0])


# ---------------------------------------------------------------- groups of tensors

class Group:
    """Tensors of a group with numpy twins; `lead` elements of padding come before each tensor's data."""

    def __init__(self, torch, xt, lengths, param="f32", grad="f32", state="f32", copy=False, lead=0, seed=0, step=0, decay=0.05, sparse=True, **cfg):
        rng = np.random.default_rng(seed)
        self.torch, self.xt, self.lengths = torch, xt, lengths
        self.s8 = state == "8bit"

        def dev(a, dtype):
            buf = torch.zeros(len(a) + lead, dtype=dtype, device="cuda")
            buf[lead:] = torch.from_numpy(a).to(dtype)
            return buf[lead:]

        pt, gt = _types(torch, param)[0], _types(torch, grad)[0]
        self.p = [dev(rng.standard_normal(n) * 0.1, pt) for n in lengths]
        self.g = [dev(rng.standard_normal(n) * rng.uniform(1e-4, 1e-1) * (rng.random(n) > (0.1 if sparse else 0)), gt) for n in lengths]
        m = [(rng.standard_normal(n) * 1e-2).astype(np.float32) * (step > 0) for n in lengths]
        v = [(rng.random(n) * 1e-3 + 1e-9).astype(np.float32) * (step > 0) for n in lengths]
        self.ms = self.vs = None
        if self.s8:
            em = [train.encode(a, np.full(len(a), 1 << 15), True) for a in m]
            ev = [train.encode(a, np.full(len(a), 1 << 15), False) for a in v]
            self.m, self.ms = [dev(a, torch.uint8) for a, _ in em], [dev(b, torch.uint8) for _, b in em]
            self.v, self.vs = [dev(a, torch.uint8) for a, _ in ev], [dev(b, torch.uint8) for _, b in ev]
        else:
            self.m, self.v = [dev(a, torch.float32) for a in m], [dev(a, torch.float32) for a in v]
        self.copy = [dev(np.zeros(n), torch.bfloat16) for n in lengths] if copy else None
        self.decay = [decay if i % 2 == 0 else 0.0 for i in range(len(lengths))]
        self.seed = cfg.get("hash_seed", 99)
        self.beta2 = cfg.get("beta2", 0.999)
        self.step = step
        self.handle = xt.xp_group_create(self.p, self.g, self.m, self.v, m_scales=self.ms, v_scales=self.vs, copies=self.copy,
                                         weight_decay=self.decay, seed=self.seed, step=step, beta2=self.beta2)
        self.report = torch.zeros(8, device="cuda")

    def close(self):
        self.xt.xp_group_destroy(self.handle)

    def states(self, i, dtype=np.float32):
        if self.s8:
            m = train.decode(self.m[i].cpu().numpy(), self.ms[i].cpu().numpy(), True)
            v = train.decode(self.v[i].cpu().numpy(), self.vs[i].cpu().numpy(), False)
            return m.astype(dtype), v.astype(dtype)
        return self.m[i].cpu().numpy().astype(dtype), self.v[i].cpu().numpy().astype(dtype)

    def twin(self, lr, scale=1.0):
        """What the next step makes of every tensor: fp32 in the formula's order (exact), and 64 bits."""
        self.step += 1
        out, pos = [], 0
        for i, n in enumerate(self.lengths):
            res = []
            for dtype in (np.float32, np.float64):
                m, v = self.states(i, dtype)
                p, g = (t.float().cpu().numpy().astype(dtype) for t in (self.p[i], self.g[i]))
                s = np.float32(scale)
                res.append(train.adamw(p, g, m, v, self.step, lr, float(np.float32(self.decay[i])), beta2=self.beta2, scale=s))
            codes = None
            if self.s8:
                hm, hv = train.rounding_bits(self.seed, self.step, range(pos, pos + n))
                codes = train.encode(res[0][1], hm, True), train.encode(res[0][2], hv, False)
            out.append((res[0], res[1], codes))
            pos += -(-n // 32) * 32
        return out

    def check(self, want):
        torch = self.torch
        for i, (f32, f64, codes) in enumerate(want):
            p = torch.from_numpy(f32[0])
            assert torch.equal(self.p[i].cpu(), p.to(self.p[i].dtype)), i
            if self.copy:
                assert torch.equal(self.copy[i].cpu(), p.bfloat16())
            if self.s8:
                for got, s, (c, e) in ((self.m[i], self.ms[i], codes[0]), (self.v[i], self.vs[i], codes[1])):
                    assert np.array_equal(s.cpu().numpy(), e), i
                    assert np.array_equal(got.cpu().numpy(), c), i
            else:
                assert np.array_equal(self.m[i].cpu().numpy(), f32[1]) and np.array_equal(self.v[i].cpu().numpy(), f32[2])
                # and against 64 bits: two products, a sum and rounded constants
                assert (np.abs(f32[1] - f64[1]) <= 5 * U * (np.abs(f64[1]) + 2 * np.abs(f32[1]) + 1e-2)).all()
                assert (np.abs(f32[2] - f64[2]) <= 8 * U * f64[2]).all()


LENGTHS = [[1], [31], [32], [33, 1, 7], [2048, 2049, 5], [100, 0, 3000, 64, 1], [8191, 8192, 8193, 20000]]


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("param,grad,copy", [("f32", "f32", False), ("f32", "f32", True), ("f32", "bf16", True), ("bf16", "bf16", False), ("bf16", "f32", False)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "x".join(map(str, v)))
def test_adamw_steps(xt, lengths, param, grad, copy, state):
    torch = torch_cuda()
    g = Group(torch, xt, lengths, param, grad, state, copy, seed=len(lengths), step=0 if copy else 41)
    for k in range(3):
        want = g.twin(1e-2 / (k + 1))
        xt.xp_adamw_step(g.handle, 1e-2 / (k + 1))
        g.check(want)
    assert xt.xp_group_get_step(g.handle) == g.step
    g.close()


@pytest.mark.parametrize("lead", [1, 3, 8])
@pytest.mark.parametrize("param,state", [("f32", "f32"), ("bf16", "8bit"), ("f32", "8bit"), ("bf16", "f32")])
def test_adamw_unaligned(xt, lead, param, state):
    torch = torch_cuda()
    g = Group(torch, xt, [5000, 77, 32], param, param, state, copy=param == "f32", lead=lead, step=7)
    want = g.twin(3e-3)
    xt.xp_adamw_step(g.handle, 3e-3)
    g.check(want)
    g.close()


def test_adamw_against_64_bits(xt):
    # p: the step's error is a few u of the step and of p; m / (sqrt(v) rs + eps) <= 40 keeps the bound simple
    torch = torch_cuda()
    g = Group(torch, xt, [30000], step=12, sparse=False)
    before = g.p[0].double().cpu().numpy()
    (f32, f64, _), = g.twin(1e-3)
    xt.xp_adamw_step(g.handle, 1e-3)
    got = g.p[0].double().cpu().numpy()
    assert (np.abs(got - f64[0]) <= 4 * U * np.abs(before) + 16 * U * np.abs(f64[0] - before) + 16 * U * 1e-3 * 2e-2 * 40).all()
    g.close()


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,lead", [([1], 0), ([5, 0, 33], 1), ([100000, 3, 8192], 0), ([4097] * 300, 0), ([700001], 3)])
def test_grad_norm(xt, grad, lengths, lead):
    # squares and a thread's sums in fp32 (each thread adds at most 8 squares per accumulator, then 8 accumulators), fp64
    # above: 20 u of the sum, half of it for the root
    torch = torch_cuda()
    g = Group(torch, xt, lengths, "f32", grad, lead=lead)
    sumsq, norm, scale = train.grad_norm([_f64(t) for t in g.g], 0.5, 1e-3)
    for _ in range(2):
        xt.xp_grad_norm(g.handle, g.report, 0.5, 1e-3)
        got = xt.xp_grad_report.from_buffer_copy(g.report.cpu().numpy().tobytes())
        assert abs(got.sumsq - sumsq) <= 20 * U * sumsq and got.nonfinite == 0
        assert abs(got.norm - norm) <= 12 * U * norm and abs(got.scale - scale) <= 14 * U * scale
    xt.xp_grad_norm(g.handle, g.report, accumulate=True)
    got = xt.xp_grad_report.from_buffer_copy(g.report.cpu().numpy().tobytes())
    assert abs(got.sumsq - 2 * sumsq) <= 40 * U * sumsq and got.scale == 1.0
    g.close()


def test_grad_norm_alone_and_nonfinite(xt):
    torch = torch_cuda()
    grads = [torch.randn(5000, device="cuda"), torch.randn(77, device="cuda")]
    h = xt.xp_group_create(None, grads)
    rep = torch.zeros(8, device="cuda")
    with pytest.raises(xt.XpError):
        xt.xp_adamw_step(h, 0.1)
    for bad in (float("inf"), float("nan"), 1e25):
        grads[1][76] = bad
        xt.xp_grad_norm(h, rep, max_norm=1.0)
        assert rep.view(torch.int32)[4].item() == 1
    other = [torch.zeros(5000, device="cuda"), torch.ones(77, device="cuda")]
    xt.xp_group_set_grads(h, other)
    xt.xp_grad_norm(h, rep)
    assert rep.view(torch.int32)[4].item() == 0 and abs(rep[2].item() - 77 ** 0.5) < 1e-5
    xt.xp_group_destroy(h)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_clipped_step_takes_the_reports_scale(xt, state):
    torch = torch_cuda()
    g = Group(torch, xt, [3000, 17], "f32", "f32", state, step=3)
    xt.xp_grad_norm(g.handle, g.report, 0.125, 1e-2)
    scale = g.report[3].item()
    assert 0 < scale < 0.125
    want = g.twin(1e-2, scale)
    xt.xp_adamw_step(g.handle, 1e-2, report=g.report, grad_scale=77.0)
    g.check(want)
    want = g.twin(1e-2, 0.25)
    xt.xp_adamw_step(g.handle, 1e-2, grad_scale=0.25)
    g.check(want)
    g.close()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_nonfinite_gradients(xt, state):
    torch = torch_cuda()
    g = Group(torch, xt, [200, 40], "f32", "f32", state, step=3)
    g.g[1][5] = float("nan")
    before = [t.clone() for t in g.p + g.m + g.v]
    xt.xp_grad_norm(g.handle, g.report)
    xt.xp_adamw_step(g.handle, 1e-2, report=g.report, skip_nonfinite=True)
    assert all(torch.equal(a, b) for a, b in zip(before, g.p + g.m + g.v))
    assert xt.xp_group_get_step(g.handle) == 3
    xt.xp_adamw_step(g.handle, 1e-2)
    # without the skip the element's weight, and in 8 bits its block's states, are NaN: no others
    p = [t.cpu().numpy() for t in g.p]
    assert np.isfinite(p[0]).all() and np.isnan(p[1][5]) and np.isnan(p[1]).sum() == 1
    m, v = g.states(1)
    assert np.isnan(m[:32]).sum() == (32 if state == "8bit" else 1) and np.isfinite(m[32:]).all() and np.isfinite(v[32:]).all()
    g.close()


def test_states_in_8_bits_follow_a_changing_gradient(xt):
    # v of a gradient of constant size: 200 steps at beta2 = 0.99 bring it from 1 to 0.25 + 0.75 * 0.99^200 = 0.3505 in
    # expectation.  One step's rounding is unbiased with a variance below (quantum / 2)^2, quantum <= v / 8; they decay
    # like the state, so the deviation is below 0.0625 sqrt(1 / (1 - 0.98)) = 0.44 of v for one element; the mean of
    # 4096 of them is within 5 / 64 of that
    torch = torch_cuda()
    n = 4096
    g = Group(torch, xt, [n], "f32", "f32", "8bit", beta2=0.99, step=0)
    v0 = train.encode(np.ones(n, np.float32), np.zeros(n, np.int64), False)
    g.v[0].copy_(torch.from_numpy(v0[0])), g.vs[0].copy_(torch.from_numpy(v0[1]))
    g.g[0].fill_(0.5)
    for _ in range(200):
        xt.xp_adamw_step(g.handle, 0.0)
    _, v = g.states(0, np.float64)
    want = 0.25 + 0.75 * 0.99 ** 200
    assert abs(v.mean() - want) < 5 / 64 * 0.44 * want
    g.close()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n,lead", [(1, 0), (33, 0), (5000, 0), (5000, 3)])
def test_state8_decode(xt, n, lead, out):
    torch = torch_cuda()
    rng = np.random.default_rng(n)
    dt = _types(torch, out)[0]

    def dev(a, t=torch.uint8):
        b = torch.zeros(len(a) + lead, dtype=t, device="cuda")
        b[lead:] = torch.from_numpy(a)
        return b[lead:]

    blocks = -(-n // 32)
    codes = [rng.integers(0, 256, n).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(40, 250, blocks).astype(np.uint8) for _ in range(2)]
    scales[0][0] = 255 if n == 33 else scales[0][0]
    mo, vo = dev(np.zeros(n), dt), dev(np.zeros(n), dt)
    xt.xp_state8_decode(dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1]), mo, vo)
    for got, c, s, signed in ((mo, codes[0], scales[0], True), (vo, codes[1], scales[1], False)):
        want = train.decode(c, s, signed)
        assert np.array_equal(_f64(got), want, equal_nan=True)
    keep = vo.clone()
    xt.xp_state8_decode(dev(codes[0]), dev(scales[0]), None, None, mo, None)
    assert torch.equal(keep, vo)


def test_set_grads_many_tensors_and_set_step(xt):
    torch = torch_cuda()
    g = Group(torch, xt, [3] * 1000, step=0)
    for t in g.g:
        t.mul_(-2)
    new = [t.clone() for t in g.g]
    old, g.g = g.g, new
    for t in old:
        t.fill_(float("nan"))
    xt.xp_group_set_grads(g.handle, new)
    xt.xp_group_set_step(g.handle, 500)
    g.step = 500
    want = g.twin(1e-2)
    xt.xp_adamw_step(g.handle, 1e-2)
    g.check(want)
    assert xt.xp_group_get_step(g.handle) == 501
    g.close()


def test_positions_past_32_bits(xt):
    # a tensor of 2^32 + 160 elements: its last ones hash, load and store at 64-bit offsets
    torch = torch_cuda()
    n, tail = (1 << 32) + 160, 192
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(n // 32, dtype=torch.uint8, device="cuda"), torch.zeros(n // 32, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(8)
    p[-tail:] = torch.from_numpy(rng.standard_normal(tail)).bfloat16().cuda()
    g[-tail:] = torch.from_numpy(rng.standard_normal(tail)).bfloat16().cuda()
    want = train.adamw(p[-tail:].float().cpu().numpy(), g[-tail:].float().cpu().numpy(), np.zeros(tail, np.float32), np.zeros(tail, np.float32), 1, 1e-2, 0.0)
    hm, hv = train.rounding_bits(5, 1, range(n - tail, n))
    h = xt.xp_group_create([p], [g], [m], [v], m_scales=[ms], v_scales=[vs], seed=5)
    xt.xp_adamw_step(h, 1e-2)
    assert torch.equal(p[-tail:].cpu(), torch.from_numpy(want[0]).bfloat16())
    for code, scale, x, hh, signed in ((m, ms, want[1], hm, True), (v, vs, want[2], hv, False)):
        c, e = train.encode(x, hh, signed)
        assert np.array_equal(code[-tail:].cpu().numpy(), c) and np.array_equal(scale[-tail // 32:].cpu().numpy(), e)
    assert not code[:-tail].any() and not p[:4096].any()
    xt.xp_group_destroy(h)


def test_a_step_in_a_graph_and_on_another_stream(xt):
    # backward, norm and step captured on a side stream: each replay is one more step, at the rate in device memory
    torch = torch_cuda()
    lengths = [1000, 1000]
    g = Group(torch, xt, lengths, step=0)
    x, dy, gamma, _ = _inputs(torch, 300, 1000, torch.bfloat16, torch.float32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    work = torch.empty(xt.xp_layernorm_workspace(300, 1000), dtype=torch.uint8, device="cuda")
    lr = torch.full((1,), 1e-2, device="cuda")
    side = torch.cuda.Stream()

    def once(stream):
        xt.xp_layernorm_forward(x, gamma, None, y, mean, rstd, stream=stream)
        xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx, g.g[0], g.g[1], work, stream=stream)
        xt.xp_grad_norm(g.handle, g.report, max_norm=0.5, stream=stream)
        xt.xp_adamw_step(g.handle, 123.0, report=g.report, lr_dev=lr, stream=stream)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(side)
    side.synchronize()
    g.step = 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        once(torch.cuda.current_stream())
    for k in range(3):
        lr.fill_(1e-2 / (k + 1))
        want = g.twin(1e-2 / (k + 1), g.report[3].item())
        graph.replay()
        torch.cuda.synchronize()
        g.check(want)
    assert xt.xp_group_get_step(g.handle) == 4
    g.close()


def test_refusals_on_the_gpu(xt):
    torch = torch_cuda()
    g = Group(torch, xt, [10])
    with pytest.raises(xt.XpError):
        xt.xp_adamw_step(g.handle, float("nan"))
    with pytest.raises(xt.XpError):
        xt.xp_adamw_step(g.handle, 0.1, skip_nonfinite=True)
    with pytest.raises(xt.XpError):
        xt.xp_grad_norm(g.handle, g.report[1:])
    with pytest.raises(xt.XpError):
        xt.xp_grad_norm(g.handle, g.report, grad_scale=float("inf"))
    assert xt._lib.xp_adamw_step(g.handle, 0.1, None, 1.0, None, 8, None) == xt.xp.XP_ERR_INVALID
    assert xt._lib.xp_group_set_grads(g.handle, (xt.ctypes.c_void_p * 1)(None), None) == xt.xp.XP_ERR_INVALID
    assert xt.xp_group_get_step(g.handle) == 0
    x = torch.randn(100, 64, device="cuda")
    s = torch.zeros(100, device="cuda")
    with pytest.raises(xt.XpError):
        xt.xp_layernorm_backward(x, x.clone(), None, s, s, torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda"),
                                 torch.empty(16, dtype=torch.uint8, device="cuda"))
    g.close()


@pytest.mark.parametrize("cols", [200, 1000, 3001, 40000])
def test_each_call_waits_for_the_one_before(xt, cols):
    # kernels may be placed while their predecessors drain: a chain in which each call reads what the call before it wrote
    # gives the same bits with and without a pause between the calls
    torch = torch_cuda()
    rows = 30

    def chain(pause):
        x, dy, gamma, beta = _inputs(torch, rows, cols, torch.float32, torch.float32)
        mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        dg, db = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
        m, v = [torch.zeros(cols, device="cuda") for _ in range(2)], [torch.zeros(cols, device="cuda") for _ in range(2)]
        spare = [torch.full((cols,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda")]
        group = xt.xp_group_create([gamma, beta], spare, m, v)
        report = torch.zeros(8, device="cuda")
        work = torch.empty(xt.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        a, b = x, torch.empty_like(x)
        out = []
        for k in range(12):
            y = torch.empty_like(x)
            dx = torch.empty_like(x)
            calls = [lambda: xt.xp_layernorm_forward(a, gamma, beta, y, mean, rstd),
                     lambda: xt.xp_layernorm_backward(dy, a, gamma, mean, rstd, dx, dg, db, work),
                     lambda: xt.xp_group_set_grads(group, [dg, db] if k % 3 else [db, dg]),
                     lambda: xt.xp_grad_norm(group, report, max_norm=0.5),
                     lambda: xt.xp_adamw_step(group, 1e-2, report=report)]
            for call in calls:
                call()
                if pause:
                    torch.cuda.synchronize()
            a, b = y, a
            out += [y, dx, report.clone()]
        torch.cuda.synchronize()
        xt.xp_group_destroy(group)
        return out + [gamma, beta, m[0], v[1]]

    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(chain(False), want))

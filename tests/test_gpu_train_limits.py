"""The training operators at the ends of their ranges, on the GPU: magnitudes far from 1, values that are not finite, and
calls that a program may make although few do."""
import numpy as np
import pytest

from oracle import train
from tests.gpu_util import torch_cuda
from tests.test_gpu_train import U, _f64, _forward_bounds, _matrix, _types, xt  # noqa: F401

pytestmark = pytest.mark.gpu

# A backward sum's depth: 16 pairs per thread and their two halves, 5 shuffle levels, up to 4 additions and 4 levels over
# a CTA's warps, 8 cluster ranks: 38; 1 / cols, its product, and the rounding of a and of x - mean come on top.
SUM_BACK = 44 * U


def _dx_bound(dy, x, gamma, mean, rstd, uo):
    """dx and what it may be off by, from float64 arrays.  With sums off by SUM_BACK of their terms' magnitudes, the two
    fused operations and their inputs off by U of what they add up (3 U each with second-order terms), d rstd (rstd s)
    by 5 U of itself, and the last product by U."""
    want, _, _ = train.layernorm_backward(dy, x, gamma, mean, rstd)
    xhat = np.abs((x - mean[:, None]) * rstd[:, None])
    a = dy if gamma is None else dy * gamma
    m1, m2 = np.abs(a).mean(1, keepdims=True), (np.abs(a) * xhat).mean(1, keepdims=True)
    inner = 6 * U * (np.abs(a) + m1 + xhat * m2) + SUM_BACK * (m1 + xhat * m2) + 5 * U * xhat * m2
    bound = inner * rstd[:, None] + 2 * U * np.abs(want)
    return want, bound + uo * (np.abs(want) + bound)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-14, 1e13, 1e15])
@pytest.mark.parametrize("rows,cols", [(306, 64), (10007, 64), (40, 200), (300, 1000), (40, 1031), (2000, 1031), (2, 9001), (3, 20000), (2, 70000)])
def test_layernorm_of_rows_of_any_size(xt, rows, cols, scale, name):
    # the powers of rstd that the definition does not have would leave fp32's range here
    torch = torch_cuda()
    dtype, uo = _types(torch, name)
    rng = np.random.default_rng(rows + cols)
    x = _matrix(torch, (rng.standard_normal((rows, cols)) + rng.standard_normal((rows, 1))) * scale, dtype)
    dy = _matrix(torch, rng.standard_normal((rows, cols)) * 0.1 + 0.02, dtype)
    gamma = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).float().cuda()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    xt.xp_layernorm_forward(x, gamma, None, y, mean, rstd, 0.0)
    xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx)
    x64, g64 = _f64(x), _f64(gamma)
    want = _forward_bounds(x64, g64, None, 0.0, uo)
    for got, ref, bound in zip((y, mean, rstd), want[:3], want[3:]):
        assert (np.abs(_f64(got) - ref) <= bound).all()
    want, bound = _dx_bound(_f64(dy), x64, g64, _f64(mean), _f64(rstd), uo)
    off = np.abs(_f64(dx) - want)
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("cols", [64, 512, 1031, 16384])
def test_gradient_of_constant_rows(xt, cols):
    # no deviation, and eps so small that rstd is 1e14: dx = rstd (a - mean a), finite
    torch = torch_cuda()
    x, dy = torch.full((3, cols), 2.0, device="cuda"), torch.randn(3, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(cols))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    xt.xp_layernorm_forward(x, None, None, y, mean, rstd, 1e-28)
    xt.xp_layernorm_backward(dy, x, None, mean, rstd, dx)
    assert torch.equal(mean, x[:, 0]) and not y.any()
    want, bound = _dx_bound(_f64(dy), _f64(x), None, _f64(mean), _f64(rstd), 0.0)
    assert (np.abs(_f64(dx) - want) <= bound).all()

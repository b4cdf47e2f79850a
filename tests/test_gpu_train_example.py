"""The data-parallel example: layer norm, the ring allreduce, the gradient norm and AdamW together.  The replicas stay
equal bit for bit, a replayed graph does what the calls do, and the training follows the same training in 64 bits."""
import os
import sys

import numpy as np
import pytest

from oracle import train as formulas
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    torch_cuda()
    from collective_transport_plane_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_virtual_ranks
    return train_virtual_ranks


@pytest.mark.parametrize("ranks,state8", [(2, False), (4, True), (8, False)])
def test_replicas_stay_equal_and_learn(example, ranks, state8):
    torch = torch_cuda()
    losses, params = example.train(ranks=ranks, steps=40, cols=96, outputs=8, rows=33, state8=state8)
    assert all(torch.equal(params[0], p) for p in params[1:])
    # the target is within the model's reach up to the tanh: a few dozen steps of 3e-3 take well over half of it away
    assert torch.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]


def test_a_replayed_step_equals_the_calls(example):
    torch = torch_cuda()
    a, pa = example.train(ranks=3, steps=12, cols=200, outputs=4, rows=17)
    b, pb = example.train(ranks=3, steps=12, cols=200, outputs=4, rows=17, replay=True)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(pa, pb))


def test_first_steps_follow_64_bits(example):
    # three steps of the same training in float64.  The step is lr * m / sqrt(v): where a gradient's error is a share e of
    # it, the step moves by about e of lr.  fp32 matrix products of 64 terms leave e near 1e-6 of a typical gradient, and
    # elements whose gradient is a thousandth of that 1e-3: so weights agree to 3 steps * lr * 1e-2 = 1e-4 everywhere,
    # and losses to 1e-4 of themselves
    torch = torch_cuda()
    ranks, cols, outputs, rows, steps, lr = 2, 64, 8, 32, 3, 3e-3
    torch.backends.cuda.matmul.allow_tf32 = False
    losses, params = example.train(ranks=ranks, steps=steps, cols=cols, outputs=outputs, rows=rows, lr=lr)
    gen = torch.Generator("cuda").manual_seed(0)
    xs = [torch.randn(rows, cols, generator=gen, device="cuda") * 2 + 0.5 for _ in range(ranks)]
    teacher = torch.randn(cols, outputs, generator=gen, device="cuda") * cols ** -0.5
    target = torch.cat([torch.tanh(torch.nn.functional.layer_norm(x, (cols,)) @ teacher) for x in xs]).double().cpu().numpy()
    x = torch.cat(xs).double().cpu().numpy()
    gen = torch.Generator("cuda").manual_seed(1)
    w = (torch.randn(outputs, cols, generator=gen, device="cuda") * cols ** -0.5).double().cpu().numpy()
    p = {"weight": w, "gamma": np.ones(cols), "beta": np.zeros(cols), "bias": np.zeros(outputs)}
    m, v = ({k: np.zeros_like(a) for k, a in p.items()} for _ in range(2))
    for t in range(1, steps + 1):
        y, mean, rstd = formulas.layernorm_forward(x, p["gamma"], p["beta"])
        err = y @ p["weight"].T + p["bias"] - target
        assert abs(losses[t - 1].item() - (err ** 2).mean()) < 1e-4 * (err ** 2).mean()
        d = 2 * err / err.size
        _, dgamma, dbeta = formulas.layernorm_backward(d @ p["weight"], x, p["gamma"], mean, rstd)
        g = {"weight": d.T @ y, "gamma": dgamma, "beta": dbeta, "bias": d.sum(0)}
        _, _, scale = formulas.grad_norm(list(g.values()), 1.0, 1.0)
        for k in p:
            p[k], m[k], v[k] = formulas.adamw(p[k], g[k], m[k], v[k], t, lr, 0.01 if k == "weight" else 0.0, scale=scale)
    flat = params[0].double().cpu().numpy()
    at = 0
    for k in ("weight", "gamma", "beta", "bias"):
        n = p[k].size
        assert np.abs(flat[at:at + n] - p[k].reshape(-1)).max() < 1e-4, k
        at += -(-n // 32) * 32

"""The distillation example: it runs, replicas stay equal, a replayed graph gives what calls give, and its gradients are
those of its formulas."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import model
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXAMPLE = os.path.join(ROOT, "examples", "distill_virtual_ranks.py")


@pytest.fixture(scope="module")
def example():
    torch_cuda()
    from collective_transport_plane_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("distill_virtual_ranks", EXAMPLE)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_calls_and_replays_agree_and_replicas_stay_equal(example):
    torch = torch_cuda()
    runs = [example.train(ranks=3, steps=6, cols=200, vocab=700, rows=90, replay=replay) for replay in (False, True)]
    for losses, params in runs:
        assert torch.isfinite(losses).all() and all(torch.equal(params[0], p) for p in params[1:])
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1][0], runs[1][1][0])


def test_gradients_are_those_of_the_layers_formulas(example):
    # The formulas in 64 bits take the numbers as the step has them in 8 bits, the gradient of the logits but once: there its
    # encoding is off by 2^-4 of each number (and 2^-10 of its block's scale, at most 2^-8 of the block's largest / 1.75).
    torch = torch_cuda()
    rows, cols, vocab, top = 70, 300, 900, 8
    r = example.Replica(cols, vocab, rows, top, 2.0, 1)
    (x, residual, ids, t), = example.batches(1, rows, cols, vocab, top, 2.0)
    dloss = torch.rand(rows, device="cuda")
    r.gradients(x, residual, ids, t, dloss, torch.cuda.current_stream())
    n = lambda a: a.double().cpu().numpy()  # noqa: E731
    codes = lambda c, s, b: model.decode(c.cpu().numpy(), s.cpu().numpy(), b)  # noqa: E731
    y, w, yt = codes(r.y8, r.sy, 1), codes(r.w8, r.sw, 128), codes(r.y8t, r.syt, 1)
    z = y @ w.T
    loss, lse = model.distill_forward(z, ids.cpu().numpy(), n(t), 2.0)
    assert np.abs(n(r.loss) - loss).max() < 1e-3
    dz = model.distill_backward(z, ids.cpu().numpy(), n(t), lse, n(dloss), 2.0)
    off = 2.0 ** -4 * np.abs(dz) + 2.0 ** -8 * np.abs(dz).max(1, keepdims=True) / 1.75 + 1e-4 * np.abs(dz).max()
    off_t = 2.0 ** -4 * np.abs(dz) + 2.0 ** -8 * np.abs(dz).max(0, keepdims=True) / 1.75 + 1e-4 * np.abs(dz).max()
    assert (np.abs(n(r.dy) - dz @ w) <= off @ np.abs(w) + 2.0 ** -7 * np.abs(dz) @ np.abs(w)).all()
    assert (np.abs(n(r.dweight) - dz.T @ yt.T) <= off_t.T @ np.abs(yt).T + 1e-4 * np.abs(dz).T @ np.abs(yt).T).all()
    # together the errors of both signs cancel: the whole gradient points the right way
    want = (dz.T @ yt.T).ravel()
    assert np.dot(n(r.dweight).ravel(), want) / np.linalg.norm(want) / np.linalg.norm(n(r.dweight)) > 0.999
    dx, dgamma = model.rmsnorm_backward(n(r.dy), n(r.h), n(r.gamma), n(r.rstd))
    assert np.abs(n(r.dgamma) - dgamma).max() <= 1e-4 * np.abs(dgamma).max() and np.abs(n(r.dx) - dx).max() <= 2.0 ** -7 * np.abs(dx).max()
    r.close()


def test_the_command_runs():
    out = subprocess.run([sys.executable, EXAMPLE, "--ranks", "2", "--steps", "3", "--replay"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "2 replicas equal" in out.stdout, out.stdout + out.stderr[-2000:]


def test_the_first_call_within_a_capture():
    # in a process of its own, every kernel first met within a capture
    code = f"""if True:
        import sys
        sys.path.insert(0, {ROOT!r})
        import torch
        import importlib.util
        spec = importlib.util.spec_from_file_location("example", {EXAMPLE!r})
        example = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(example)
        r = example.Replica(256, 3000, 600, 4, 1.0, 1)
        (x, residual, ids, t), = example.batches(1, 600, 256, 3000, 4, 1.0)
        dloss = torch.ones(600, device="cuda")
        torch.cuda.synchronize()
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            r.gradients(x, residual, ids, t, dloss, st)
        g.replay()
        torch.cuda.synchronize()
        got = r.grads.clone()
        r.gradients(x, residual, ids, t, dloss, torch.cuda.current_stream())
        torch.cuda.synchronize()
        print(torch.equal(got, r.grads), bool(got.abs().sum() > 0))"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.stdout.split() == ["True", "True"], out.stdout + out.stderr[-2000:]

"""Data-parallel training on virtual ranks of one GPU, through the library's own calls.

Every rank holds a replica of a small regression model, layer norm then a linear map, and its share of the batch.
A step on each rank: layer norm forward and backward (xp_train), the two matrix products of the linear map (torch), all
gradients in one flat fp32 buffer; then one ring allreduce of those buffers (xp), the gradients' global norm and the
clipped AdamW step (xp_train).  The host waits for nothing within a step.  As every rank computes the same from the same
sums, the replicas stay equal bit for bit.

    python examples/train_virtual_ranks.py --ranks 4 --steps 50 [--state8] [--replay]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from collective_transport_plane_gb300 import xp, xp_train  # noqa: E402

BLOCK = xp_train.XP_STATE8_BLOCK


class Replica:
    """One rank's model: its tensors are views of flat buffers, each padded to the 8-bit states' blocks."""

    def __init__(self, cols, outputs, rows, state8, seed):
        shapes = [("weight", (outputs, cols)), ("gamma", (cols,)), ("beta", (cols,)), ("bias", (outputs,))]
        sizes = [-(-torch.Size(s).numel() // BLOCK) * BLOCK for _, s in shapes]
        total = sum(sizes)
        self.params, self.grads = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
        state = torch.uint8 if state8 else torch.float32
        m, v = torch.zeros(total, dtype=state, device="cuda"), torch.zeros(total, dtype=state, device="cuda")
        m_scale, v_scale = (torch.zeros(total // BLOCK, dtype=torch.uint8, device="cuda") if state8 else None for _ in range(2))
        self.kept = (m, v, m_scale, v_scale)     # the group names their memory
        self.p, self.g, at = {}, {}, 0
        lists = {k: [] for k in ("p", "g", "m", "v", "ms", "vs")}
        for (name, shape), size in zip(shapes, sizes):
            n = torch.Size(shape).numel()
            self.p[name], self.g[name] = self.params[at:at + n].view(shape), self.grads[at:at + n].view(shape)
            for key, flat in (("p", self.params), ("g", self.grads), ("m", m), ("v", v)):
                lists[key].append(flat[at:at + n])
            if state8:
                blocks = slice(at // BLOCK, (at + n + BLOCK - 1) // BLOCK)
                lists["ms"].append(m_scale[blocks])
                lists["vs"].append(v_scale[blocks])
            at += size
        self.p["gamma"].fill_(1.0)
        gen = torch.Generator("cuda").manual_seed(seed)
        self.p["weight"].copy_(torch.randn(outputs, cols, generator=gen, device="cuda") * cols ** -0.5)
        self.group = xp_train.xp_group_create(
            lists["p"], lists["g"], lists["m"], lists["v"], m_scales=lists["ms"] or None, v_scales=lists["vs"] or None,
            weight_decay=[0.01 if name == "weight" else 0.0 for name, _ in shapes], seed=seed)
        self.report = torch.zeros(8, device="cuda")
        self.y, self.dx = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
        self.mean, self.rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        self.work = torch.empty(xp_train.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")

    def gradients(self, x, target, batch, stream):
        """This rank's part of the loss, mean over `batch` rows of the whole job, and of its gradients."""
        p, g = self.p, self.g
        xp_train.xp_layernorm_forward(x, p["gamma"], p["beta"], self.y, self.mean, self.rstd, stream=stream)
        err = torch.addmm(p["bias"], self.y, p["weight"].t()) - target
        d = err * (2.0 / (batch * target.shape[1]))
        torch.mm(d.t(), self.y, out=g["weight"])
        torch.sum(d, 0, out=g["bias"])
        xp_train.xp_layernorm_backward(d @ p["weight"], x, p["gamma"], self.mean, self.rstd, self.dx, g["gamma"], g["beta"],
                                       self.work, stream=stream)
        return err.square().sum() / (batch * target.shape[1])

    def close(self):
        xp_train.xp_group_destroy(self.group)


def train(ranks=4, steps=50, cols=512, outputs=64, rows=256, state8=False, replay=False, lr=3e-3, max_norm=1.0, seed=0):
    """Losses per step (a tensor on the GPU), and the replicas' weights."""
    gen = torch.Generator("cuda").manual_seed(seed)
    xs = [torch.randn(rows, cols, generator=gen, device="cuda") * 2 + 0.5 for _ in range(ranks)]
    teacher = torch.randn(cols, outputs, generator=gen, device="cuda") * cols ** -0.5
    targets = [torch.tanh(torch.nn.functional.layer_norm(x, (cols,)) @ teacher) for x in xs]
    replicas = [Replica(cols, outputs, rows, state8, seed + 1) for _ in range(ranks)]
    ring = xp.xp_ring_create(ranks, 2, 4, 64 << 10)
    losses = torch.zeros(steps, device="cuda")
    lr_now, at = torch.full((1,), lr, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        stream = torch.cuda.current_stream()
        loss = sum(r.gradients(x, t, ranks * rows, stream) for r, x, t in zip(replicas, xs, targets))
        losses.index_copy_(0, at, loss.reshape(1))
        at.add_(1)
        flat = [r.grads for r in replicas]
        xp.xp_ring_allreduce_virtual(ring, flat, flat, flat[0].numel(), xp.XP_F32, stream)
        for r in replicas:
            xp_train.xp_grad_norm(r.group, r.report, max_norm=max_norm, stream=stream)
            xp_train.xp_adamw_step(r.group, lr, report=r.report, lr_dev=lr_now, skip_nonfinite=True, stream=stream)

    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = None
        for k in range(steps):
            with torch.cuda.stream(side):
                if graph is None:
                    step()
                else:
                    graph.replay()
            if replay and k == 0:    # the first step, outside a capture, sets the kernels up
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
        side.synchronize()
        status, report = xp.xp_ring_status(ring, True)
        if status != xp.XP_OK:
            raise RuntimeError(f"the ring reports {xp.xp_status_string(status)} at rank and channel {report.channel}")
        return losses, [r.params.clone() for r in replicas]
    finally:
        torch.cuda.synchronize()
        xp.xp_ring_destroy(ring)
        for r in replicas:
            r.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--state8", action="store_true", help="keep the AdamW states in 8 bits")
    ap.add_argument("--replay", action="store_true", help="capture a step in a CUDA graph and replay it")
    a = ap.parse_args()
    losses, params = train(a.ranks, a.steps, state8=a.state8, replay=a.replay)
    same = all(torch.equal(params[0], p) for p in params[1:])
    for k in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {k:4d}  loss {losses[k].item():.6f}")
    print(f"last       loss {losses[-1].item():.6f}; {a.ranks} replicas {'equal' if same else 'DIFFER'}")


if __name__ == "__main__":
    main()

"""Data-parallel distillation in 8 bits on virtual ranks of one GPU, through the library's own calls.

Every rank holds a replica of a model's last layer, a root-mean-square norm of hidden states and their residual and a linear
map to the vocabulary, and its share of the batch with a teacher's top logits.  A step on each rank (xp_model): the weight in
8 bits, the norm with an output in 8 bits, the product, the loss and its gradient, the gradient in 8 bits along both axes,
the two products of the backward pass, the norm's backward pass.  Then one ring allreduce of the fp32 gradients (xp), their
global norm and the clipped AdamW step (xp_train).  The host waits for nothing within a step, and the replicas stay equal bit
for bit.

    python examples/distill_virtual_ranks.py --ranks 4 --steps 50 [--replay]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from collective_transport_plane_gb300 import xp, xp_model, xp_train  # noqa: E402

BLOCK = xp_model.XP_BLOCK8


def codes8(rows, cols):
    """A matrix in 8 bits: codes whose rows are multiples of 128 bytes apart, and the scales of `block_rows` 1."""
    up = lambda n, k: -(-n // k) * k  # noqa: E731
    codes = torch.zeros(rows, up(cols, 128), dtype=torch.uint8, device="cuda")[:, :cols]
    blocks = -(-cols // BLOCK)
    return codes, torch.zeros(rows, up(blocks, 4), dtype=torch.uint8, device="cuda")[:, :blocks]


class Replica:
    """One rank's last layer, its gradients in one flat fp32 buffer, and the buffers of a step."""

    def __init__(self, cols, vocab, rows, top, temperature, seed):
        self.cols, self.vocab, self.T = cols, vocab, temperature
        empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        bf16, n = torch.bfloat16, vocab * cols
        self.params, self.grads = torch.zeros(n + cols, device="cuda"), torch.zeros(n + cols, device="cuda")
        self.weight, self.gamma = self.params[:n].view(vocab, cols), self.params[n:]
        self.dweight, self.dgamma = self.grads[:n].view(vocab, cols), self.grads[n:]
        gen = torch.Generator("cuda").manual_seed(seed)
        self.weight.copy_(torch.randn(vocab, cols, generator=gen, device="cuda") * cols ** -0.5)
        self.gamma.fill_(1.0)
        self.m, self.v = torch.zeros_like(self.params), torch.zeros_like(self.params)
        cut = lambda t: [t[:n], t[n:]]  # noqa: E731
        self.group = xp_train.xp_group_create(cut(self.params), cut(self.grads), cut(self.m), cut(self.v), weight_decay=[0.01, 0.0])
        self.report = torch.zeros(8, device="cuda")
        # the weight and its transpose share codes and scales of blocks of 128 x 128
        (self.w8, sw), (self.w8t, swt) = codes8(vocab, cols), codes8(cols, vocab)
        self.sw, self.swt = sw[:-(-vocab // BLOCK)], swt[:-(-cols // BLOCK)]
        (self.y8, self.sy), (self.y8t, self.syt) = codes8(rows, cols), codes8(cols, rows)
        (self.dz8, self.sdz), (self.dz8t, self.sdzt) = codes8(rows, vocab), codes8(vocab, rows)
        self.h, self.y, self.dy, self.dx = (empty(rows, cols, dtype=bf16) for _ in range(4))
        self.rstd, self.loss, self.lse, self.logits = empty(rows), empty(rows), empty(rows), empty(rows, vocab)
        self.work = empty(max(16, xp_model.xp_rmsnorm_workspace(rows, cols)), dtype=torch.uint8)

    def gradients(self, x, residual, ids, teacher, dloss, stream):
        """This rank's part of the gradients of sum(dloss * loss); the losses are in self.loss."""
        xm = xp_model
        xm.xp_block8_encode(self.weight, self.w8, self.sw, self.w8t, self.swt, block_rows=BLOCK, stream=stream)
        xm.xp_rmsnorm_forward(x, self.gamma, self.y, residual, self.h, self.rstd, self.y8, self.sy, stream=stream)
        xm.xp_matmul8(self.y8, self.sy, self.w8, self.sw, self.logits, b_block_rows=BLOCK, stream=stream)
        xm.xp_distill_forward(self.logits, ids, teacher, self.loss, self.lse, self.T, stream=stream)
        xm.xp_distill_backward(self.logits, ids, teacher, self.lse, dloss, self.logits, self.T, stream=stream)   # in their place
        xm.xp_block8_encode(self.logits, self.dz8, self.sdz, self.dz8t, self.sdzt, stream=stream)
        xm.xp_block8_encode(self.y, codes_t=self.y8t, scales_t=self.syt, stream=stream)
        xm.xp_matmul8(self.dz8, self.sdz, self.w8t, self.swt, self.dy, b_block_rows=BLOCK, stream=stream)
        xm.xp_matmul8(self.dz8t, self.sdzt, self.y8t, self.syt, self.dweight, stream=stream)
        xm.xp_rmsnorm_backward(self.dy, self.h, self.gamma, self.rstd, self.dx, self.dgamma, self.work, stream=stream)

    def close(self):
        xp_train.xp_group_destroy(self.group)


def batches(ranks, rows, cols, vocab, top, temperature, seed=0):
    """Each rank's hidden states, residual, and a random teacher's top logits; some entries name no token."""
    gen = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    teacher = normal(cols, vocab) * 2 * cols ** -0.5
    out = []
    for _ in range(ranks):
        x, r = normal(rows, cols).bfloat16(), normal(rows, cols).bfloat16()
        values, ids = torch.nn.functional.rms_norm((x + r).float(), (cols,)).matmul(teacher).topk(top, 1)
        ids[torch.rand(rows, top, generator=gen, device="cuda") < 0.05] = -1
        out.append((x, r, ids.int(), values.contiguous()))
    return out


def train(ranks=4, steps=50, cols=512, vocab=2000, rows=256, top=16, temperature=2.0, replay=False, lr=2e-3, max_norm=1.0, seed=0):
    """Mean losses per step (a tensor on the GPU), and the replicas' weights."""
    data = batches(ranks, rows, cols, vocab, top, temperature, seed)
    replicas = [Replica(cols, vocab, rows, top, temperature, seed + 1) for _ in range(ranks)]
    ring = xp.xp_ring_create(ranks, 2, 4, 64 << 10)
    dloss = torch.full((rows,), 1.0 / (ranks * rows), device="cuda")
    losses, at = torch.zeros(steps, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        stream = torch.cuda.current_stream()
        for r, (x, residual, ids, teacher) in zip(replicas, data):
            r.gradients(x, residual, ids, teacher, dloss, stream)
        losses.index_copy_(0, at, sum((r.loss * dloss).sum() for r in replicas).reshape(1))
        at.add_(1)
        flat = [r.grads for r in replicas]
        xp.xp_ring_allreduce_virtual(ring, flat, flat, flat[0].numel(), xp.XP_F32, stream)
        for r in replicas:
            xp_train.xp_grad_norm(r.group, r.report, max_norm=max_norm, stream=stream)
            xp_train.xp_adamw_step(r.group, lr, report=r.report, skip_nonfinite=True, stream=stream)

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
        if xp_model.xp_matmul8_status() != xp.XP_OK:
            raise RuntimeError("a product gave up a wait")
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
    ap.add_argument("--replay", action="store_true", help="capture a step in a CUDA graph and replay it")
    a = ap.parse_args()
    losses, params = train(a.ranks, a.steps, replay=a.replay)
    same = all(torch.equal(params[0], p) for p in params[1:])
    for k in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {k:4d}  loss {losses[k].item():.6f}")
    print(f"last       loss {losses[-1].item():.6f}; {a.ranks} replicas {'equal' if same else 'DIFFER'}")


if __name__ == "__main__":
    main()

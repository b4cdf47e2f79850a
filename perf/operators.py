"""Cases for measuring the training operators next to the ring allreduce: layer norm forward and backward,
the global gradient norm with its clip factor, and the AdamW step over many tensors.

Many tensors live in flat buffers, each tensor padded with zeros to a multiple of 32 elements, as a
data-parallel program keeps them so that one allreduce moves all gradients.  `own` chooses between the
plain torch form of each operator and the calls of `collective_transport_plane_gb300.xp_train`."""
import math
import weakref

import numpy as np
import torch

own = False

BLOCK = 32                       # elements of one scale of an 8-bit state
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.999, 1e-8, 0.1, 3e-4
MAX_NORM = 1.0
LN_EPS = 1e-5
SEED8 = 20231                    # of the 8-bit states' rounding
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the weights of a small probe or head: the call's latency counts
        {"name": "adamw_tiny", "op": "adamw", "tensors": 6, "numel": 5001, "param": "f32", "grad": "f32", "state": "f32",
         "copy": False, "clip": False, "step": 1},
        # a block's weights after the allreduce of fp32 gradients: clipped by the global norm, bf16 working copy
        {"name": "adamw_clip_copy", "op": "adamw", "tensors": 148, "numel": 28_000_003, "param": "f32", "grad": "f32",
         "state": "f32", "copy": True, "clip": True, "step": 100},
        # one rank's 256 MiB of the ring benchmark, as weights
        {"name": "adamw_ring_rank", "op": "adamw", "tensors": 2, "numel": 1 << 26, "param": "f32", "grad": "f32",
         "state": "f32", "copy": False, "clip": False, "step": 5000},
        # a small adapter kept in bf16 with 8-bit states
        {"name": "adamw8_small", "op": "adamw", "tensors": 20, "numel": 300_000, "param": "bf16", "grad": "bf16",
         "state": "8bit", "copy": False, "clip": False, "step": 3},
        # a rank's shard of a large model in bf16 with 8-bit states, clipped
        {"name": "adamw8_large", "op": "adamw", "tensors": 60, "numel": 100_000_000, "param": "bf16", "grad": "bf16",
         "state": "8bit", "copy": False, "clip": True, "step": 700},
        # the norm of an adapter's gradients, and of one replica's
        {"name": "norm_small", "op": "norm", "tensors": 40, "numel": 200_001, "grad": "bf16"},
        {"name": "norm_large", "op": "norm", "tensors": 300, "numel": 1 << 27, "grad": "f32"},
        # a few tokens at a time
        {"name": "ln_fwd_small", "op": "ln_fwd", "rows": 7, "cols": 1000, "type": "bf16", "weight": "f32", "pad": 0},
        # a batch of 8 sequences of 2048 tokens
        {"name": "ln_fwd_batch", "op": "ln_fwd", "rows": 16384, "cols": 4096, "type": "bf16", "weight": "bf16", "pad": 0},
        # a small model's batch
        {"name": "ln_bwd_small", "op": "ln_bwd", "rows": 64, "cols": 768, "type": "f32", "weight": "f32", "pad": 0},
        # odd rows and columns inside wider rows: nothing is aligned
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 9973, "cols": 1031, "type": "bf16", "weight": "f32", "pad": 6},
        # a large batch of wide rows
        {"name": "ln_bwd_batch", "op": "ln_bwd", "rows": 24576, "cols": 5120, "type": "bf16", "weight": "f32", "pad": 0},
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["adamw", "adamw", "norm", "ln_fwd", "ln_bwd", "ln_bwd"])
    if op in ("adamw", "norm"):
        numel = between(3000, 90_000_000)
        case = {"op": op, "tensors": min(between(1, 400), numel // 64), "numel": numel, "grad": rng.choice(["f32", "bf16"])}
        if op == "adamw":
            param = rng.choice(["f32", "bf16"])
            case |= {"param": param, "state": rng.choice(["f32", "8bit"]), "copy": param == "f32" and rng.random() < 0.5,
                     "clip": rng.random() < 0.5, "step": between(1, 20000)}
        return case
    cols = between(33, 66_000)
    cols = cols // 64 * 64 + 32 if rng.random() < 0.5 else cols | 1
    rows = between(1, min(65_536, max(2, 100_000_000 // cols)))
    return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["f32", "bf16"]), "weight": rng.choice(["f32", "bf16"]),
            "pad": rng.choice([0, 0, 0, 8, 6, 1])}


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """The tensors' lengths, the same for every seed: the first half weights of ragged sizes, the rest short vectors."""
    n, rs = case["tensors"], np.random.RandomState(case["tensors"])
    w = np.exp(rs.normal(0, 1, n))
    w[n - n // 2:] *= 1e-3
    return np.maximum(1, np.floor(w / w.sum() * case["numel"])).astype(np.int64)


def _layout(case):
    """(lengths, offsets, flat length, where the tensors without weight decay begin)."""
    n = _lengths(case)
    padded = -(-n // BLOCK) * BLOCK
    off = np.concatenate([[0], np.cumsum(padded)])
    first_vector = case["tensors"] - case["tensors"] // 2
    return n, off[:-1], int(off[-1]), int(off[first_vector])


def _flat_mask(n, off, total):
    """1 where the flat buffer holds an element of a tensor, 0 in its padding."""
    mark = torch.zeros(total + 1, dtype=torch.int8, device="cuda")
    mark[torch.from_numpy(off).cuda()] += 1
    mark.index_add_(0, torch.from_numpy(off + n).cuda(), torch.full((len(n),), -1, dtype=torch.int8, device="cuda"))
    return mark.cumsum(0, dtype=torch.int8)[:-1]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case)
    if case["op"] in ("adamw", "norm"):
        n, off, total, split = _layout(case)
        mask = _flat_mask(n, off, total)
        # gradients differ in size from tensor to tensor, and some weights got none
        size = torch.from_numpy(np.exp(np.random.RandomState(seed % (1 << 31)).normal(-6, 1, len(n))).astype(np.float32)).cuda()
        each = torch.repeat_interleave(size, torch.from_numpy(-(-n // BLOCK) * BLOCK).cuda(), output_size=total)
        g = normal(total) * each * mask
        g *= torch.rand(total, generator=gen, device="cuda") > 0.02
        s |= {"grad_flat": g.to(TYPES[case["grad"]]), "off": off, "n": n, "split": split,
              "report": torch.zeros(8, device="cuda")}
        s |= {"norm": s["report"][2:3], "scale": s["report"][3:4], "bad": s["report"].view(torch.int32)[4:5]}
        if case["op"] == "adamw":
            s["p"] = (normal(total) * 0.02 * mask).to(TYPES[case["param"]])
            started = 0.0 if case["step"] == 1 else 1.0
            m = normal(total) * each * mask * (0.3 * started)
            v = (normal(total).square() * 0.5 + 0.5) * each.square() * mask * started
            if case["state"] == "8bit":
                half = torch.full((1,), 1 << 19, dtype=torch.int32, device="cuda")
                s["m"], s["m_scale"] = _encode(m, half, True)
                s["v"], s["v_scale"] = _encode(v, half, False)
                s["m_out"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
                s["v_out"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
            else:
                s["m"], s["v"] = m, v
            s["copy_flat"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
            s["t"] = case["step"] - 1
        if own:
            s["group"] = _plan(s)
        return s
    rows, cols, dt, wt = case["rows"], case["cols"], TYPES[case["type"]], TYPES[case["weight"]]

    def rowwise(values):
        wide = torch.zeros(rows, cols + case["pad"], dtype=dt, device="cuda")
        wide[:, :cols] = values
        return wide[:, :cols]

    x = normal(rows, cols) * (0.5 + torch.rand(rows, 1, generator=gen, device="cuda") * 2) + normal(rows, 1)
    s["x"] = rowwise(x)
    s["gamma"] = (1 + 0.1 * normal(cols)).to(wt)
    s["beta"] = (0.1 * normal(cols) + 0.05).to(wt)
    if case["op"] == "ln_fwd":
        s |= {"y": torch.empty(rows, cols, dtype=dt, device="cuda"), "mean": torch.empty(rows, device="cuda"),
              "rstd": torch.empty(rows, device="cuda")}
        return s
    s["dy"] = rowwise(normal(rows, cols) * 0.01 + 0.003)
    s["mean"], s["rstd"] = _statistics(s["x"])
    s |= {"dx": torch.empty(rows, cols, dtype=dt, device="cuda"), "dgamma": torch.empty(cols, device="cuda"),
          "dbeta": torch.empty(cols, device="cuda")}
    if own:
        from collective_transport_plane_gb300 import xp_train
        s["work"] = torch.empty(xp_train.xp_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    return s


class _Handle:
    """A group of tensors' handle, destroyed with the state that holds it."""

    def __init__(self, xp_train, handle):
        self.handle = handle
        weakref.finalize(self, xp_train.xp_group_destroy, handle)


def _plan(s):
    from collective_transport_plane_gb300 import xp_train

    def views(name):
        flat = s.get(name)
        return None if flat is None else [flat[o:o + k] for o, k in zip(s["off"].tolist(), s["n"].tolist())]

    def scales(name):
        flat = s.get(name)
        return None if flat is None else [flat[o // BLOCK:(o + k + BLOCK - 1) // BLOCK] for o, k in zip(s["off"].tolist(), s["n"].tolist())]

    if s["op"] == "norm":
        return _Handle(xp_train, xp_train.xp_group_create(None, views("grad_flat")))
    first_vector = s["tensors"] - s["tensors"] // 2
    return _Handle(xp_train, xp_train.xp_group_create(
        views("p"), views("grad_flat"), views("m"), views("v"), m_scales=scales("m_scale"), v_scales=scales("v_scale"),
        copies=views("copy_flat"), weight_decay=[DECAY if i < first_vector else 0.0 for i in range(s["tensors"])],
        beta1=BETA1, beta2=BETA2, eps=EPS, seed=SEED8, step=s["t"]))


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        from collective_transport_plane_gb300 import xp_train
        if s["op"] == "ln_fwd":
            xp_train.xp_layernorm_forward(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], LN_EPS)
            return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        if s["op"] == "ln_bwd":
            xp_train.xp_layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"], s["work"])
            return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
        group = s["group"].handle
        if s["op"] == "norm":
            xp_train.xp_grad_norm(group, s["report"], max_norm=MAX_NORM)
            return {"norm": s["norm"], "scale": s["scale"], "bad": s["bad"]}
        if s["clip"]:
            xp_train.xp_grad_norm(group, s["report"], max_norm=MAX_NORM)
        xp_train.xp_adamw_step(group, LR, report=s["report"] if s["clip"] else None)
        out = {"p": s["p"], "copy": s["copy_flat"]}
        if s["clip"]:
            out["norm"] = s["norm"]
        if s["state"] == "f32":
            return out | {"m": s["m"], "v": s["v"]}
        xp_train.xp_state8_decode(s["m"], s["m_scale"], s["v"], s["v_scale"], s["m_out"], s["v_out"])
        return out | {"m": s["m_out"], "v": s["v_out"]}
    if s["op"] == "ln_fwd":
        return _ln_fwd(s)
    if s["op"] == "ln_bwd":
        return _ln_bwd(s)
    if s["op"] == "norm":
        return _norm(s["grad_flat"])
    return _adamw(s)


def _statistics(x):
    x = x.float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    return mean, 1 / ((d * d).sum(1) / x.shape[1] + LN_EPS).sqrt()


def _ln_fwd(s):
    mean, rstd = _statistics(s["x"])
    y = (s["x"].float() - mean[:, None]) * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _ln_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    a = dy * s["gamma"].float()
    c1 = a.sum(1, keepdim=True) / a.shape[1]
    c2 = (a * xhat).sum(1, keepdim=True) / a.shape[1]
    return {"dx": ((a - c1 - xhat * c2) * rstd).to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _norm(grad):
    g = grad.float()
    norm = (g * g).sum().sqrt().reshape(1)
    return {"norm": norm, "scale": torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm)), "bad": (~torch.isfinite(norm)).int()}


# An 8-bit state: 32 elements share a scale byte E, the biased exponent of their largest magnitude in fp32, and a
# magnitude is an exponent and 3 mantissa bits: code c > 0 stands for the fp32 number whose bits are (c + 8 E - K) << 20.
# v takes all 8 bits (K = 247), m 7 bits and a sign (K = 119); c = 0 is zero, E = 255 a block that is not finite.
# Rounding is stochastic: 20 bits, a function of the seed, the step and the element's position, are added below the cut.
# A positive v never becomes 0, so that no step divides by eps alone where m is left.

def _decode(code, scale, signed):
    c, e = code.int().view(-1, BLOCK), scale.int()[:, None]
    mag = c & 127 if signed else c
    x = ((mag + 8 * e - (119 if signed else 247)).clamp(min=0) << 20).view(torch.float32)
    x = torch.where(mag == 0, torch.zeros_like(x), x)
    x = torch.where(c > 127, -x, x) if signed else x
    return torch.where(e == 255, torch.full_like(x, float("nan")), x).view(-1)


def _encode(x, noise, signed):
    bits = x.abs().view(torch.int32)
    e = (bits >> 23).view(-1, BLOCK).amax(1)
    c = ((bits + noise) >> 20).view(-1, BLOCK) - (8 * e - (119 if signed else 247))[:, None]
    c = c.clamp(0 if signed else 1, 127 if signed else 255).view(-1)
    c = torch.where(bits == 0, torch.zeros_like(c), c)
    c = c + 128 * ((x < 0) & (c > 0)) if signed else c
    return c.to(torch.uint8), e.to(torch.uint8)


def _noise(total, t, device):
    """The rounding bits of m and of v: a 32-bit mix of the position and of a key that the seed and the step give."""
    key = _mix((SEED8 * 0x8ED88009 + _mix(t & 0xFFFFFFFF)) & 0xFFFFFFFF)
    pos = torch.arange(total, device=device)
    h = _mix(((pos & 0xFFFFFFFF) * 0x8ED88009 + (pos >> 32) * 0xB86D3E2F + key) & 0xFFFFFFFF)
    return ((h >> 16 << 4) + 8).int(), (((h & 0xFFFF) << 4) + 8).int()


def _mix(x):
    x = ((x ^ (x >> 16)) * 0xDDF15BA9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xE31B8755) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _adamw(s):
    s["t"] = t = s["t"] + 1
    f = np.float32
    alpha = float(f(LR) * f(1 / (1 - BETA1 ** t)))
    rs = float(f(1 / math.sqrt(1 - BETA2 ** t)))
    out = {}
    g = s["grad_flat"].float()
    if s["clip"]:
        clip = _norm(s["grad_flat"])
        out["norm"] = clip["norm"]
        g = g * clip["scale"]
    bits8 = s["state"] == "8bit"
    m = _decode(s["m"], s["m_scale"], True) if bits8 else s["m"]
    v = _decode(s["v"], s["v_scale"], False) if bits8 else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * (1 - BETA2) * g
    step = (m * alpha) / (v.sqrt() * rs + EPS)
    p, k = s["p"].float(), s["split"]
    keep = float(f(1) - f(LR) * f(DECAY))
    p = torch.cat([p[:k] * keep, p[k:]]) - step
    s["p"].copy_(p)
    if bits8:
        noise_m, noise_v = _noise(len(p), t, p.device)
        s["m"], s["m_scale"] = _encode(m, noise_m, True)
        s["v"], s["v_scale"] = _encode(v, noise_v, False)
        out |= {"m": _decode(s["m"], s["m_scale"], True).bfloat16(), "v": _decode(s["v"], s["v_scale"], False).bfloat16()}
    else:
        s["m"], s["v"] = m, v
        out |= {"m": m, "v": v}
    return out | {"p": s["p"], "copy": p.bfloat16() if s["copy"] else None}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] in ("adamw", "norm"):
        n = int(_lengths(case).sum())
        sg = size[case["grad"]]
        if case["op"] == "norm":
            return {"bytes": n * sg + 12, "flops": 2 * n}
        # read and write the weights, read the gradients, read and write both states, write the copy; 8-bit states are
        # also written out as bf16 values
        states = 16 if case["state"] == "f32" else 4 + 4 / BLOCK + 4
        return {"bytes": n * (2 * size[case["param"]] + sg + states + (2 if case["copy"] else 0)),
                "flops": n * (15 + (2 if case["clip"] else 0))}
    r, c, sx, sw = case["rows"], case["cols"], size[case["type"]], size[case["weight"]]
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * r * c * sx + 2 * c * sw + 8 * r, "flops": 8 * r * c}
    return {"bytes": 3 * r * c * sx + c * sw + 8 * c + 8 * r, "flops": 14 * r * c}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + LN_EPS).rsqrt()
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "ln_bwd":
        # through the transpose of the Jacobian: projections off the constant and off xhat; from the statistics it is given
        dy, r = s["dy"].double(), s["rstd"].double()
        xhat = (s["x"].double() - s["mean"].double()[:, None]).mul_(r[:, None])
        dgamma, dbeta = torch.einsum("rc,rc->c", dy, xhat), dy.sum(0)
        a = dy.mul_(s["gamma"].double())
        along = torch.einsum("rc,rc->r", a, xhat) / case["cols"]
        a.sub_(a.mean(1, keepdim=True)).addcmul_(xhat, along[:, None], value=-1.0).mul_(r[:, None])
        return {"dx": a, "dgamma": dgamma, "dbeta": dbeta}
    g = s["grad_flat"].double()
    norm = torch.linalg.vector_norm(g).reshape(1)
    if case["op"] == "norm":
        return {"norm": norm, "scale": (MAX_NORM / norm).clamp(max=1.0), "bad": None}
    t = case["step"]
    if case["clip"]:
        g *= (MAX_NORM / norm).clamp(max=1.0)
    bits8 = case["state"] == "8bit"
    m = _value64(s["m"], s["m_scale"], 128) if bits8 else s["m"].double()
    v = _value64(s["v"], s["v_scale"], 256) if bits8 else s["v"].double()
    m.lerp_(g, 1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    p = s["p"].double()
    p[: s["split"]] *= 1 - LR * DECAY
    p -= LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    if bits8:
        h = _hash64(len(p), t)
        m, v = _round64(m, (h >> 16).double(), 128), _round64(v, (h & 0xFFFF).double(), 256)
    return {"p": p, "copy": p if case["copy"] else None, "m": m, "v": v, **({"norm": norm} if case["clip"] else {})}


def _value64(code, scale, codes):
    """What codes stand for: `codes` magnitudes, 8 to a power of two, the last of them the power above E's."""
    c = code.view(-1, BLOCK).double()
    sign = torch.where(c >= codes, -1.0, 1.0)
    mag = torch.remainder(c, codes)
    # fp32 bits (mag + 8 E - K) << 20 with K = codes - 9: exponent (mag + 8 E - K) / 8 - 127, mantissa the rest / 8
    at = mag + 8 * scale.double()[:, None] - (codes - 9)
    power = torch.floor(at / 8)
    x = torch.ldexp(1 + (at / 8 - power), power - 127)
    return (torch.where(mag == 0, 0.0, x) * sign).view(-1)


def _round64(x, noise16, codes):
    """The value that each number is rounded to: down to a step of its power of two after adding its noise, in steps."""
    _, power = torch.frexp(x)
    power = power - 1
    top = torch.where(x == 0, -126, power).view(-1, BLOCK).amax(1, keepdim=True)
    quantum = torch.ldexp(torch.ones_like(x), power - 3)
    y = torch.floor(x.abs() / quantum + (noise16 + 0.5) / 65536) * quantum
    least = torch.ldexp(torch.full_like(top, 1.25, dtype=torch.float64), top - (codes - 8) // 8)  # code 1
    y = y.view(-1, BLOCK)
    if codes == 128:
        y = torch.where(y < least, 0.0, y)
    else:
        y = torch.where(x.view(-1, BLOCK) > 0, torch.maximum(y, least), y)
    return y.view(-1).where(x != 0, 0.0) * torch.sign(x)


def _hash64(total, t):
    """The same 32-bit mix, on numpy's wrapping unsigned integers."""
    def mix(x):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0xDDF15BA9)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0xE31B8755)
        return x ^ (x >> np.uint32(16))

    key = mix(np.array([SEED8], np.uint32) * np.uint32(0x8ED88009) + mix(np.array([t], np.uint32)))
    h = mix(np.arange(total, dtype=np.uint32) * np.uint32(0x8ED88009) + key)
    return torch.from_numpy(h.astype(np.int64)).cuda()

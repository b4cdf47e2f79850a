"""Cases for measuring the operators of a layer that trains and serves in 8 bits: the root-mean-square norm with the
residual's addition and an output in 8 bits, the encoding of matrices in 8 bits by blocks of 128, the product of such
matrices, and the loss that distils a teacher's top logits, with its gradient.

`own` chooses between the plain torch form of each operator and the calls of
`collective_transport_plane_gb300.xp_model`.  What is held in 8 bits (a code of 4 exponent and 3 mantissa bits, times
2^(E - 127) for the scale byte E of its block) is returned as the values it stands for."""
import math

import torch

own = False

BLOCK = 128                      # elements of one scale along the axis that a product sums over
EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token's norm on its way into a product: latency
        {"name": "rms_fwd_token", "op": "rms_fwd", "rows": 1, "cols": 4096, "type": "bf16", "weight": "bf16", "residual": True,
         "wide": False, "pad": 0},
        # a batch of 8 sequences of 2048 tokens in training: the sum, the norm for the backward pass, the norm in 8 bits
        {"name": "rms_fwd_batch", "op": "rms_fwd", "rows": 16384, "cols": 4096, "type": "bf16", "weight": "f32", "residual": True,
         "wide": True, "pad": 0},
        # odd rows of an odd length, nothing aligned
        {"name": "rms_bwd_odd", "op": "rms_bwd", "rows": 4099, "cols": 1031, "type": "f32", "weight": "f32", "residual": False, "pad": 0},
        # a large batch of wide rows, with the gradient that comes along the residual
        {"name": "rms_bwd_batch", "op": "rms_bwd", "rows": 16384, "cols": 5120, "type": "bf16", "weight": "f32", "residual": True, "pad": 0},
        # a ragged batch's gradient, as both products of a backward pass read it
        {"name": "encode_odd", "op": "encode", "rows": 1001, "cols": 1000, "type": "f32", "block_rows": 1, "pad": 0},
        # a batch's activations or gradient, both forms
        {"name": "encode_batch", "op": "encode", "rows": 16384, "cols": 4096, "type": "bf16", "block_rows": 1, "pad": 0},
        # a token through a weight
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 4096, "out": "bf16", "b_block_rows": 128, "add": False},
        # a weight's gradient added up over an odd number of tokens
        {"name": "product_grad", "op": "product", "m": 4096, "n": 5120, "k": 16001, "out": "f32", "b_block_rows": 1, "add": True},
        # a batch through a wide weight
        {"name": "product_batch", "op": "product", "m": 8192, "n": 16384, "k": 4096, "out": "bf16", "b_block_rows": 128, "add": False},
        # the loss of a few rows
        {"name": "distill_fwd_few", "op": "distill_fwd", "rows": 61, "vocab": 32000, "type": "f32", "top": 8, "temperature": 2.0},
        # a batch's loss
        {"name": "distill_fwd_batch", "op": "distill_fwd", "rows": 8192, "vocab": 32000, "type": "bf16", "top": 64, "temperature": 1.0},
        # its gradient over a vocabulary whose rows are not aligned
        {"name": "distill_bwd_odd", "op": "distill_bwd", "rows": 4095, "vocab": 50257, "type": "bf16", "top": 50, "temperature": 2.0},
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def uneven(n):
        return rng.choice([n | 1, n, -(-n // 16) * 16, -(-n // 128) * 128])

    op = rng.choice(["rms_fwd", "rms_bwd", "encode", "product", "product", "distill_fwd", "distill_bwd"])
    if op == "product":
        n, k = uneven(between(64, 16000)), uneven(between(64, 16000))
        m = between(1, min(16000, max(1, (1 << 38) // (n * k))))
        m = m if m < 64 else uneven(m)
        out = rng.choice(["bf16", "f32"])
        return {"op": op, "m": m, "n": n, "k": k, "out": out, "b_block_rows": rng.choice([1, 128]), "add": out == "f32" and rng.random() < 0.5}
    kind = rng.choice(["f32", "bf16"])
    if op in ("distill_fwd", "distill_bwd"):
        vocab = uneven(between(1000, 160_000))
        rows = between(1, min(16_384, 200_000_000 // vocab))
        return {"op": op, "rows": rows, "vocab": vocab, "type": kind, "top": between(1, 128), "temperature": rng.choice([1.0, 2.0, 0.7])}
    cols = uneven(between(64, 20_000))
    rows = between(1, min(65_536, 60_000_000 // cols))
    case = {"op": op, "rows": rows, "cols": cols, "type": kind, "pad": rng.choice([0, 0, 0, 16, 3])}
    if op == "encode":
        return case | {"block_rows": rng.choice([1, 1, 128])}
    case |= {"weight": rng.choice(["f32", "bf16"]), "residual": rng.random() < 0.7}
    return case | ({"wide": rng.random() < 0.5} if op == "rms_fwd" else {})


# ---------------------------------------------------------------- inputs

def _ceil(a, b):
    return -(-a // b)


def _codes(rows, cols):
    """A matrix of codes whose rows are a multiple of 16 bytes apart, and what lies behind a row's end."""
    return torch.zeros(rows, _ceil(cols, 16) * 16, dtype=torch.uint8, device="cuda")[:, :cols]


def _scales(rows, cols):
    """Its scales: a byte for each 128 columns, rows a multiple of 4 bytes apart."""
    return torch.zeros(rows, _ceil(_ceil(cols, BLOCK), 4) * 4, dtype=torch.uint8, device="cuda")[:, :_ceil(cols, BLOCK)]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s, op = dict(case), case["op"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # rows of different size with a few large channels; weights, or for a gradient the other operand's columns
        a = normal(m, k) * (0.3 + 2 * uniform(m, 1)) * torch.where(uniform(1, k) < 0.01, 20.0, 1.0)
        b = normal(n, k) * (k ** -0.5 if case["b_block_rows"] == 128 else 1e-3)
        s["a"], s["a_scales"], s["b"], s["b_scales"] = _codes(m, k), _scales(m, k), _codes(n, k), _scales(_ceil(n, case["b_block_rows"]), k)
        for name, x, block_rows in (("a", a, 1), ("b", b, case["b_block_rows"])):
            codes, scales = _encode(x, block_rows)
            s[name].copy_(codes)
            s[name + "_scales"].copy_(scales)
        s["c"] = torch.empty(m, n, dtype=TYPES[case["out"]], device="cuda")
        s["c"].copy_(normal(m, n) * 0.1)
        return s
    dt = TYPES[case["type"]]
    if op in ("distill_fwd", "distill_bwd"):
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        s["logits"] = (normal(rows, vocab) * 2.5).to(dt)
        teacher = s["logits"].float() + normal(rows, vocab)
        values, ids = teacher.topk(top, 1)
        # some rows have fewer entries, and padded ones have none
        left = torch.where(uniform(rows, 1) < 0.1, (uniform(rows, 1) * (top + 1)).floor(), float(top))
        s["ids"] = torch.where(torch.arange(top, device="cuda") < left, ids, -1).int()
        s["teacher"] = values
        s["loss"], s["lse"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if op == "distill_bwd":
            s["lse"] = torch.logsumexp(s["logits"].double() / case["temperature"], 1).float()
            s["dloss"] = (0.5 + uniform(rows)) / rows
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    rows, cols = case["rows"], case["cols"]

    def rowwise(values=None):
        wide = torch.zeros(rows, cols + case["pad"], dtype=dt, device="cuda")
        if values is not None:
            wide[:, :cols] = values
        return wide[:, :cols]

    x = normal(rows, cols) * (0.5 + 2 * uniform(rows, 1)) * torch.where(uniform(1, cols) < 0.01, 10.0, 1.0)
    s["x"] = rowwise(x)
    if op == "encode":
        b = case["block_rows"]
        s["codes"], s["scales"] = _codes(rows, cols), _scales(_ceil(rows, b), cols)
        s["codes_t"], s["scales_t"] = _codes(cols, rows), _scales(_ceil(cols, b), rows)
        s["out"], s["out_t"] = (torch.empty(*shape, dtype=torch.bfloat16, device="cuda") for shape in ((rows, cols), (cols, rows)))
        return s
    s["gamma"] = (1 + 0.1 * normal(cols)).to(TYPES[case["weight"]])
    if op == "rms_fwd":
        s["residual_in"] = rowwise(normal(rows, cols)) if case["residual"] else None
        s["added"] = rowwise() if case["residual"] else None
        s["y"] = rowwise() if case["wide"] else None
        s["rstd"] = torch.empty(rows, device="cuda")
        s["y8"], s["y8_scales"] = _codes(rows, cols), _scales(rows, cols)
        s["y8_out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        return s
    s["dy"] = rowwise(normal(rows, cols) * 0.01)
    s["dadded"] = rowwise(normal(rows, cols) * 0.01) if case["residual"] else None
    s["rstd"] = _rstd(s["x"].float())
    s["dx"], s["dgamma"] = rowwise(), torch.empty(cols, device="cuda")
    if own:
        from collective_transport_plane_gb300 import xp_model
        s["work"] = torch.empty(xp_model.xp_rmsnorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "product":
        c = _decode(s["a"], s["a_scales"], 1) @ _decode(s["b"], s["b_scales"], s["b_block_rows"]).t()
        s["c"].copy_(s["c"] + c if s["add"] else c)
        return {"c": s["c"]}
    if op == "distill_fwd":
        loss, lse = _distill_fwd(s["logits"], s["ids"], s["teacher"], s["temperature"])
        return {"loss": loss, "lse": lse}
    if op == "distill_bwd":
        return {"dlogits": _distill_bwd(s["logits"], s["ids"], s["teacher"], s["lse"], s["dloss"], s["temperature"])}
    if op == "encode":
        b = s["block_rows"]
        codes, scales = _encode(s["x"].float(), b)
        codes_t, scales_t = _encode(s["x"].float().t(), b)
        return {"out": _decode(codes, scales, b).bfloat16(), "out_t": _decode(codes_t, scales_t, b).bfloat16()}
    x, gamma = s["x"].float(), s["gamma"].float()
    if op == "rms_fwd":
        added = (x + s["residual_in"].float()).to(s["x"].dtype) if s["residual"] else None
        h = added.float() if s["residual"] else x
        rstd = _rstd(h)
        y = h * rstd[:, None] * gamma
        codes, scales = _encode(y, 1)
        return {"added": added, "y": y.to(s["x"].dtype) if s["wide"] else None, "rstd": rstd, "y8": _decode(codes, scales, 1).bfloat16()}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat, a = x * rstd, dy * gamma
    dx = (a - xhat * ((a * xhat).sum(1, keepdim=True) / a.shape[1])) * rstd
    if s["residual"]:
        dx = dx + s["dadded"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0)}


def _own(s):
    from collective_transport_plane_gb300 import xp_model
    op = s["op"]
    if op == "product":
        xp_model.xp_matmul8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["c"], b_block_rows=s["b_block_rows"], accumulate=s["add"])
        return {"c": s["c"]}
    if op == "distill_fwd":
        xp_model.xp_distill_forward(s["logits"], s["ids"], s["teacher"], s["loss"], s["lse"], s["temperature"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "distill_bwd":
        xp_model.xp_distill_backward(s["logits"], s["ids"], s["teacher"], s["lse"], s["dloss"], s["dlogits"], s["temperature"])
        return {"dlogits": s["dlogits"]}
    if op == "encode":
        b = s["block_rows"]
        xp_model.xp_block8_encode(s["x"], s["codes"], s["scales"], s["codes_t"], s["scales_t"], block_rows=b)
        xp_model.xp_block8_decode(s["codes"], s["scales"], s["out"], block_rows=b)
        xp_model.xp_block8_decode(s["codes_t"], s["scales_t"], s["out_t"], block_rows=b)
        return {"out": s["out"], "out_t": s["out_t"]}
    if op == "rms_fwd":
        xp_model.xp_rmsnorm_forward(s["x"], s["gamma"], s["y"], residual=s["residual_in"], added=s["added"], rstd=s["rstd"], y8=s["y8"],
                                    y8_scales=s["y8_scales"], eps=EPS)
        xp_model.xp_block8_decode(s["y8"], s["y8_scales"], s["y8_out"])
        return {"added": s["added"], "y": s["y"], "rstd": s["rstd"], "y8": s["y8_out"]}
    xp_model.xp_rmsnorm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["work"], dadded=s["dadded"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _rstd(x):
    return 1 / ((x * x).sum(1) / x.shape[1] + EPS).sqrt()


# 8 bits with a scale for each block: 128 columns of one row (block_rows 1) or of 128 rows (block_rows 128) share the byte E, the least
# with max |x| <= 448 * 2^(E - 127) (255: the block is not finite); a code is x / 2^(E - 127) rounded to 4 exponent and 3 mantissa bits, ties to even.

def _power(e):
    """2^(e - 127) of scale bytes in fp32."""
    e = e.int()
    return torch.where(e == 0, 0x00400000, e << 23).view(torch.float32)


def _padded(x, block_rows):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK, 0, -x.shape[0] % block_rows))


def _encode(x, block_rows):
    rows, cols = x.shape
    x = _padded(x, block_rows).unflatten(1, (-1, BLOCK)).unflatten(0, (-1, block_rows))       # blocks of rows, rows, blocks, columns
    bits = x.abs().amax((1, 3)).view(torch.int32)
    e = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=0)
    e = torch.where(bits >= 0x7F800000, 255, e)
    codes = (x * _power((254 - e).clamp(min=0))[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where((e == 255)[:, None, :, None], 127, codes)
    return codes.flatten(2).flatten(0, 1)[:rows, :cols], e.to(torch.uint8)


def _decode(codes, scales, block_rows):
    rows, cols = codes.shape
    p = torch.where(scales == 255, float("nan"), _power(scales))
    p = p.repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else p
    return codes.contiguous().view(torch.float8_e4m3fn).float() * p.repeat_interleave(BLOCK, 1)[:, :cols]


def _teacher(ids, teacher, vocab, temperature):
    """(p, log p, where an entry counts, where a row has any): the softmax of the teacher's logits over the entries that name a token."""
    there = (ids >= 0) & (ids < vocab)
    u = torch.where(there, teacher.float() / temperature, -math.inf)
    top = u.amax(1, keepdim=True)
    any_ = top > -math.inf
    w = torch.where(any_, (u - top).exp(), 0.0)
    total = w.sum(1, keepdim=True)
    return w / total, u - top - total.log(), there & (u > -math.inf), any_


def _distill_fwd(logits, ids, teacher, temperature):
    z = logits.float() / temperature
    top = z.amax(1, keepdim=True)
    lse = (z - top).exp().sum(1, keepdim=True).log() + top
    p, logp, there, any_ = _teacher(ids, teacher, z.shape[1], temperature)
    at = z.gather(1, ids.clamp(0, z.shape[1] - 1).long())
    loss = torch.where(there, p * (logp - (at - lse)), 0.0).sum(1) * temperature ** 2
    return torch.where(any_[:, 0], loss, 0.0), torch.where(any_, lse, 0.0)[:, 0]


def _distill_bwd(logits, ids, teacher, lse, dloss, temperature):
    z = logits.float() / temperature
    p, _, there, any_ = _teacher(ids, teacher, z.shape[1], temperature)
    d = torch.where(any_, (z - lse[:, None]).exp(), 0.0)
    d.scatter_add_(1, ids.clamp(0, z.shape[1] - 1).long(), torch.where(there, -p, 0.0))
    return (d * (dloss * temperature)[:, None]).to(logits.dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = _ceil(k, BLOCK)
        return {"bytes": (m + n) * k + (m + _ceil(n, case["b_block_rows"])) * blocks + m * n * size[case["out"]] * (2 if case["add"] else 1),
                "flops": 2 * m * n * k}
    rows, t = case["rows"], size[case["type"]]
    if case["op"] in ("distill_fwd", "distill_bwd"):
        v = rows * case["vocab"]
        back = case["op"] == "distill_bwd"
        return {"bytes": (2 if back else 1) * v * t + rows * case["top"] * 8 + 8 * rows, "flops": 4 * v}
    n, blocks = rows * case["cols"], rows * _ceil(case["cols"], BLOCK)
    if case["op"] == "encode":
        # both forms are written, and written out again as bf16 values
        b = case["block_rows"]
        scales = _ceil(rows, b) * _ceil(case["cols"], BLOCK) + _ceil(case["cols"], b) * _ceil(rows, BLOCK)
        return {"bytes": n * (t + 2 + 4) + scales, "flops": 6 * n}
    w = case["cols"] * size[case["weight"]]
    if case["op"] == "rms_fwd":
        # read x, and the residual; write the sum, the norm, and the norm in 8 bits, which is also written out as bf16 values
        return {"bytes": n * (t * (1 + (2 if case["residual"] else 0) + (1 if case["wide"] else 0)) + 1 + 2) + blocks + w + 4 * rows, "flops": 7 * n}
    return {"bytes": n * t * (4 if case["residual"] else 3) + w + 4 * case["cols"] + 4 * rows, "flops": 9 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "product":
        if case["m"] * case["n"] * case["k"] > 8e11:
            return None
        a, b = _value64(s["a"], s["a_scales"], 1), _value64(s["b"], s["b_scales"], case["b_block_rows"])
        return {"c": torch.addmm(s["c"].double(), a, b.t(), beta=1.0 if case["add"] else 0.0)}
    if op in ("distill_fwd", "distill_bwd"):
        t, vocab = case["temperature"], case["vocab"]
        ids = s["ids"].long()
        logq = torch.log_softmax(s["logits"].double() / t, 1)
        teacher = torch.where(ids < 0, -math.inf, s["teacher"].double() / t)
        some = (ids >= 0).any(1)
        p = torch.where(some[:, None], torch.softmax(teacher, 1), 0.0)
        if op == "distill_fwd":
            at = logq.gather(1, ids.clamp(min=0))
            kl = torch.where(p > 0, torch.special.xlogy(p, p) - p * at, 0.0).sum(1)
            lse = torch.logsumexp(s["logits"].double() / t, 1)
            return {"loss": t * t * kl, "lse": torch.where(some, lse, 0.0)}
        # from the log-sum-exp it is given; entries that name no token go to a column behind the others
        d = torch.zeros(case["rows"], vocab + 1, dtype=torch.float64, device="cuda")
        d[:, :vocab] = torch.exp(s["logits"].double() / t - s["lse"].double()[:, None]) * some[:, None]
        d.scatter_add_(1, torch.where(ids < 0, vocab, ids), -p)
        return {"dlogits": d[:, :vocab] * (t * s["dloss"].double())[:, None]}
    x = s["x"].double()
    if op == "encode":
        b = case["block_rows"]
        return {"out": _round64(x, b), "out_t": _round64(x.t(), b)}
    gamma = s["gamma"].double()
    if op == "rms_fwd":
        added = x + s["residual_in"].double() if case["residual"] else None
        # the norm is that of the sum as it is stored
        h = added.to(s["x"].dtype).double() if case["residual"] else x
        rstd = (torch.linalg.vector_norm(h, dim=1).square() / case["cols"] + EPS).rsqrt()
        y = torch.einsum("rc,r,c->rc", h, rstd, gamma)
        return {"added": added, "y": y if case["wide"] else None, "rstd": rstd, "y8": _round64(y, 1)}
    # through the Jacobian's transpose: the projection off xhat, from the statistic it is given
    dy, rstd = s["dy"].double(), s["rstd"].double()
    dgamma = torch.einsum("rc,rc,r->c", dy, x, rstd)
    a = dy.mul_(gamma)
    along = torch.einsum("rc,rc->r", a, x) * rstd ** 3 / case["cols"]
    dx = torch.addcmul(a * rstd[:, None], x, along[:, None], value=-1.0)
    return {"dx": dx + s["dadded"].double() if case["residual"] else dx, "dgamma": dgamma}


def _two64(p):
    """2^p in fp64, put together from its bits (a power computed on a GPU need not be exact)."""
    return ((p.long() + 1023) << 52).view(torch.float64)


def _value64(codes, scales, block_rows):
    """What codes stand for, by their fields: (-1)^s 2^(e - 7) (1 + f / 8), 2^-6 f / 8 where e is 0."""
    c = codes.long()
    e, f = c >> 3 & 15, (c & 7).double()
    mag = torch.where(e == 0, f / 512, (8 + f) * _two64(e - 10))
    rows, cols = torch.arange(c.shape[0], device="cuda") // block_rows, torch.arange(c.shape[1], device="cuda") // BLOCK
    return torch.where(c >= 128, -mag, mag) * _two64(scales.long()[rows][:, cols] - 127)


def _round64(x, block_rows):
    """The values that the elements of a finite matrix are rounded to."""
    blocks = _padded(x, block_rows).unflatten(1, (-1, BLOCK)).unflatten(0, (-1, block_rows))
    m, p = torch.frexp(blocks.abs().amax((1, 3), keepdim=True))            # max |x| = m 2^p, 1/2 <= m < 1
    power = torch.where(m > 0.875, p - 8, p - 9).clamp(min=-127)
    _, p = torch.frexp(blocks)
    quantum = torch.maximum(p - 1, power - 6) - 3                          # a step's power of two
    out = torch.round(blocks * _two64(-quantum)) * _two64(quantum)
    return out.flatten(2).flatten(0, 1)[: x.shape[0], : x.shape[1]]

"""The training operators at the ends of their ranges, on the GPU: magnitudes far from 1, values that are not finite, and
calls that a program may make although few do."""
import threading
import time

import numpy as np
import pytest

from oracle import train
from tests.gpu_util import torch_cuda
from tests.test_gpu_train import U, Group, _f64, _forward_bounds, _matrix, _types, xt  # noqa: F401

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


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n,lead", [(5000, 0), (5000, 3), (100, 0)])
@pytest.mark.parametrize("param,state", [("f32", "f32"), ("bf16", "f32"), ("f32", "8bit"), ("bf16", "8bit")])
def test_a_second_moment_that_is_not_finite(xt, param, state, n, lead, value):
    # gradient and m are 0: over a NaN the weight is NaN, over an infinity it stays, whole turns of a CTA or not
    torch = torch_cuda()
    g = Group(torch, xt, [n], param, param, state, lead=lead, step=3, decay=0.0)
    g.g[0].zero_()
    g.m[0].zero_()
    bad = [37, n - 1]
    if state == "8bit":
        if value == float("inf"):
            g.vs[0][[b // 32 for b in bad]], g.v[0][bad] = 254, 255    # the code beyond fp32's largest number
        else:
            g.vs[0][[b // 32 for b in bad]] = 255
    else:
        g.v[0][bad] = value
    before = g.p[0].float().cpu().numpy()
    (f32, _, _), = g.twin(1e-2)
    xt.xp_adamw_step(g.handle, 1e-2)
    got = g.p[0].float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(f32[0])) and np.isnan(got[bad]).all() == (value != float("inf"))
    assert np.array_equal(got[~np.isnan(got)], before[~np.isnan(got)])
    g.close()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("param,state", [("f32", "f32"), ("f32", "8bit"), ("bf16", "8bit")])
def test_gradients_that_are_not_finite(xt, param, state, value):
    # two steps, in whole turns and at the tensor's end: an element's own weight first; in 8 bits its block's states are
    # lost with it, and every other block's codes are what they would be
    torch = torch_cuda()
    n, bad = 5000, [5, 2048 + 77, 4999]
    g = Group(torch, xt, [n], param, param, state, step=3)
    lost = np.zeros(n, bool)
    lost[bad] = True
    blocks = np.unique(np.array(bad) // 32)
    for k in range(2):
        g.g[0][bad] = value if k == 0 else 0.25
        (f32, _, codes), = g.twin(1e-2)
        xt.xp_adamw_step(g.handle, 1e-2)
        got = g.p[0].float().cpu().numpy()
        assert np.array_equal(np.isnan(got), lost)
        want = torch.from_numpy(f32[0]).to(g.p[0].dtype).float().numpy()
        assert np.array_equal(got, want, equal_nan=True)
        if state == "8bit":
            for code, scale, (c, e) in ((g.m[0], g.ms[0], codes[0]), (g.v[0], g.vs[0], codes[1])):
                scale, code = scale.cpu().numpy(), code.cpu().numpy()
                assert (scale[blocks] == 255).all()
                fine = np.ones(len(e), bool)
                fine[blocks] = False
                assert np.array_equal(scale[fine], e[fine]) and np.array_equal(code[np.repeat(fine, 32)[:n]], c[np.repeat(fine, 32)[:n]])
            lost[np.repeat(np.isin(np.arange(len(fine)), blocks), 32)[:n]] = True
    g.close()


def test_step_counts_that_would_wrap(xt):
    torch = torch_cuda()
    g = Group(torch, xt, [100], step=7)
    for step in (-1, (1 << 64) - 1, xt.XP_GROUP_MAX_STEP + 1):
        with pytest.raises(xt.XpError):
            xt.xp_group_set_step(g.handle, step)
    assert xt.xp_group_get_step(g.handle) == 7
    xt.xp_group_set_step(g.handle, xt.XP_GROUP_MAX_STEP)
    g.step = xt.XP_GROUP_MAX_STEP
    want = g.twin(1e-2)
    xt.xp_adamw_step(g.handle, 1e-2)
    g.check(want)
    g.close()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (8, 64), (9, 65), (10000, 64), (300, 1000), (310, 1031), (2, 9001), (3, 20000)])
def test_layernorm_of_side_by_side_columns(xt, rows, cols, name):
    # matrices that are columns of one buffer, in every order, give what matrices of their own give
    torch = torch_cuda()
    dtype, _ = _types(torch, name)
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    x, dy = (torch.randn(rows, cols, device="cuda", generator=gen).to(dtype) for _ in range(2))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    xt.xp_layernorm_forward(x, None, None, y, mean, rstd)
    xt.xp_layernorm_backward(dy, x, None, mean, rstd, dx)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (2, 0, 3, 1)):
        wide = torch.full((rows, 4 * cols), 7.0, dtype=dtype, device="cuda")
        xw, dyw, yw, dxw = (wide[:, k * cols:(k + 1) * cols] for k in order)
        xw.copy_(x)
        dyw.copy_(dy)
        xt.xp_layernorm_forward(xw, None, None, yw, mean, rstd)
        assert torch.equal(yw, y) and torch.equal(xw, x) and torch.equal(dyw, dy) and (dxw == 7).all()
        xt.xp_layernorm_backward(dyw, xw, None, mean, rstd, dxw)
        assert torch.equal(dxw, dx) and torch.equal(yw, y) and torch.equal(xw, x) and torch.equal(dyw, dy)


def test_one_row_in_place_at_any_stride(xt):
    torch = torch_cuda()
    x = torch.randn(1, 500, device="cuda")
    y = torch.empty_like(x)
    xt.xp_layernorm_forward(x, None, None, y.as_strided((1, 500), (7, 1)))
    xt.xp_layernorm_forward(x, None, None, x.as_strided((1, 500), (7, 1)))
    assert torch.equal(x, y)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("n,largest,lead", [(33, 1.8e19, 0), (100001, 1e19, 0), (100001, 1e19, 1), (12_000_001, 1e18, 0), (21_000_000, 7e17, 0)])
def test_norm_of_finite_gradients_up_to_the_limit(xt, grad, n, largest, lead):
    # every square is in fp32's range, the sum of a few is not.  As for ordinary sizes: 20 u of the sum, half of it and
    # 2 u for the root
    torch = torch_cuda()
    gen = torch.Generator("cuda").manual_seed(n)
    t = (torch.rand(n + lead, device="cuda", generator=gen) * 0.5 + 0.5).mul_(largest).to(_types(torch, grad)[0])[lead:]
    t[::2].neg_()
    group, report = xt.xp_group_create(None, [t]), torch.zeros(8, device="cuda")
    xt.xp_grad_norm(group, report, max_norm=1.0)
    sumsq = float(t.double().square().sum())
    got = xt.xp_grad_report.from_buffer_copy(report.cpu().numpy().tobytes())
    assert got.nonfinite == 0 and abs(got.sumsq - sumsq) <= 20 * U * sumsq
    assert abs(got.norm - sumsq ** 0.5) <= 12 * U * sumsq ** 0.5 and abs(got.scale * sumsq ** 0.5 - 1) <= 14 * U
    # and what is not finite still shows
    for bad in (float("nan"), -float("inf"), 2e19):
        keep = t[n // 2].clone()
        t[n // 2] = bad
        xt.xp_grad_norm(group, report, max_norm=1.0)
        t[n // 2] = keep
        assert report.view(torch.int32)[4].item() == 1
    xt.xp_group_destroy(group)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("n", [100, 5000, 9_000_001])
def test_norm_names_what_is_not_finite(xt, grad, n):
    # infinities give an infinite norm, a NaN anywhere a NaN, beside ordinary elements or ones whose squares only add up
    # to an infinity in fp32
    torch = torch_cuda()
    t = torch.ones(n, device="cuda").to(_types(torch, grad)[0])
    group, report = xt.xp_group_create(None, [t]), torch.zeros(8, device="cuda")
    inf, nan = float("inf"), float("nan")
    for fill in (1.0, 1.7e19):
        for where, want in (({}, None), ({0: inf}, inf), ({n - 1: -inf}, inf), ({n // 2: inf, n // 3: inf}, inf), ({n - 1: nan}, nan),
                            ({0: inf, n - 1: nan}, nan), ({0: nan, 1: inf}, nan), ({k: inf for k in range(0, n, max(1, n // 50))}, inf)):
            t.fill_(fill)
            for k, value in where.items():
                t[k] = value
            xt.xp_grad_norm(group, report, max_norm=1.0)
            norm = report[2].item()
            assert report.view(torch.int32)[4].item() == (want is not None)
            if want is None:
                exact = t[0].double().item() * n ** 0.5
                assert abs(norm - exact) <= 12 * U * exact
            else:
                assert norm == want or norm != norm and want != want
    xt.xp_group_destroy(group)


def test_reading_the_step_count_leaves_a_capture_as_it_is(xt):
    torch = torch_cuda()
    g = Group(torch, xt, [100])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        xt.xp_adamw_step(g.handle, 1e-2, stream=stream)
        with pytest.raises(xt.XpError) as refused:
            xt.xp_group_get_step(g.handle, stream)
        assert refused.value.status == xt.xp.XP_ERR_INVALID
    assert xt.xp_group_get_step(g.handle) == 0
    for k in range(3):
        want = g.twin(1e-2)
        graph.replay()
        torch.cuda.synchronize()
        g.check(want)
    assert xt.xp_group_get_step(g.handle, stream) == 3
    g.close()


def test_calls_of_several_threads(xt):
    # four threads, each on its own stream, with rows of lengths that want different amounts of shared memory of the same
    # kernel: every call is made, and gives what it gives alone
    torch = torch_cuda()
    rows, failed, made = 153, [], []

    def inputs(cols):
        gen = torch.Generator("cuda").manual_seed(cols)
        x, dy = (torch.randn(rows, cols, device="cuda", generator=gen).bfloat16() for _ in range(2))
        return dy, x, None, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"), torch.empty_like(x)

    def calls(args, stream, until):
        n = 0
        while time.monotonic() < until and not failed:
            try:
                for _ in range(50):
                    xt.xp_layernorm_backward(*args, stream=stream)
            except xt.XpError as e:
                failed.append(str(e))
            stream.synchronize()
            n += 50
        made.append(n)

    for backs in ((6144, 8192, 7168, 8192), (12000, 16384, 12288, 16384)):
        all_args, streams = [inputs(c) for c in backs], [torch.cuda.Stream() for _ in backs]
        torch.cuda.synchronize()
        until = time.monotonic() + 3.0
        threads = [threading.Thread(target=calls, args=(a, s, until)) for a, s in zip(all_args, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed, failed[0]
        for a in all_args:
            alone = torch.empty_like(a[-1])
            xt.xp_layernorm_backward(*a[:-1], alone)
            assert torch.equal(alone, a[-1])
    assert len(made) == 8 and min(made) > 0


def _states8_step(torch, xt, n, seed, p, g, m, v, lr, eps, beta2=0.999, step=41):
    """The weights that one step with 8-bit states makes of fp32 arrays, and what the same program in fp32 does."""
    half = np.full(n, 1 << 15)
    (cm, sm), (cv, sv) = train.encode(m, half, True), train.encode(v, half, False)
    t = [torch.from_numpy(a).cuda() for a in (p, g, cm, sm, cv, sv)]
    group = xt.xp_group_create([t[0]], [t[1]], [t[2]], [t[4]], m_scales=[t[3]], v_scales=[t[5]], seed=seed, step=step, eps=eps, beta2=beta2)
    xt.xp_adamw_step(group, lr)
    xt.xp_group_destroy(group)
    m, v = train.decode(cm, sm, True).astype(np.float32), train.decode(cv, sv, False).astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        return t[0].cpu().numpy(), train.adamw(p, g, m, v, step + 1, lr, 0.0, eps=eps, beta2=beta2)[0]


@pytest.mark.parametrize("m_power", [-130, -115, -100, -90, -60, 0, 45, 60, 110])
@pytest.mark.parametrize("v_power", [-110, -95, -60, -20, 0, 35, 45, 90, 110])
def test_steps_of_8_bit_states_at_any_magnitude(xt, m_power, v_power):
    # the weights are 0, so that every bit of the quotient shows: the fp32 program's, also where the quotient, its
    # remainder or its denominator is near the ends of fp32's range
    torch = torch_cuda()
    n = 1 << 14
    rng = np.random.default_rng(100000 + 200 * m_power + v_power)
    g = (rng.standard_normal(n) * 2.0 ** min(m_power, 62)).astype(np.float32)
    g[rng.random(n) < 0.1] = 0
    m = (rng.standard_normal(n) * 2.0 ** (m_power + rng.integers(-3, 4, n))).astype(np.float32)
    m[rng.random(n) < 0.1] = 0
    v = ((rng.random(n) + 0.125) * 2.0 ** (v_power + rng.integers(-3, 4, n))).astype(np.float32)
    for eps in (1e-45, 1e-8, 1.0, 1e20, 1e30, 3e38):
        for lr in (1e-3, 0.5, 0.0):
            got, want = _states8_step(torch, xt, n, 5, np.zeros(n, np.float32), g, m, v, lr, eps)
            assert np.array_equal(got, want, equal_nan=True), (eps, lr, int((got != want).sum()))


@pytest.mark.parametrize("seed", range(4))
def test_quotients_and_roots_of_8_bit_states(xt, seed):
    # 4 million pairs with random significands and magnitudes, as ordinary training has them and beyond
    torch = torch_cuda()
    n = 1 << 22
    rng = np.random.default_rng(seed)
    spread = (6, 20, 40, 60)[seed]
    g = (rng.standard_normal(n) * 2.0 ** rng.uniform(-spread, spread / 4, n)).astype(np.float32)
    m = (rng.standard_normal(n) * 2.0 ** rng.uniform(-spread, spread / 4, n)).astype(np.float32)
    v = (rng.random(n) * 2.0 ** rng.uniform(-spread, spread / 4, n) + 1e-30).astype(np.float32)
    for p in (np.zeros(n, np.float32), rng.standard_normal(n).astype(np.float32)):
        got, want = _states8_step(torch, xt, n, 5, p, g, m, v, 3e-4, 1e-8)
        assert np.array_equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(20000, 256, 0), (20000, 512, 0), (10000, 1024, 0), (9973, 1031, 6), (40000, 95, 0), (40000, 96, 0), (40000, 96, 1), (9729, 8, 0),
                                           (30001, 64, 0), (3000, 2080, 0), (2999, 4097, 0), (1300, 8192, 0), (700, 12000, 0), (611, 12001, 0), (400, 40001, 0),
                                           (170, 66000, 0), (153, 300, 0), (7, 5000, 0)])
def test_weight_gradients_add_every_row_once(xt, rows, cols, pad, name):
    # small whole numbers, mean 0 and rstd 1: every product and sum is exact (at most 32 * 40000 < 2^24), in whatever order,
    # so a row left out or taken twice, in any of the layouts, turns or tails, shows in the column's last bit
    torch = torch_cuda()
    dtype, _ = _types(torch, name)
    rng = np.random.default_rng(rows + cols)
    x, dy = (_matrix(torch, rng.integers(-k, k + 1, (rows, cols)).astype(np.float64), dtype, pad) for k in (4, 8))
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    gamma, dx = torch.ones(cols, dtype=dtype, device="cuda"), torch.empty_like(x)
    start = torch.from_numpy(rng.integers(-9, 10, (2, cols)).astype(np.float32)).cuda()
    dgamma, dbeta = start[0].clone(), start[1].clone()
    work = torch.full((xt.xp_layernorm_workspace(rows, cols),), 255, dtype=torch.uint8, device="cuda")
    want = (dy.double() * x.double()).sum(0).float(), dy.double().sum(0).float()
    xt.xp_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, work)
    assert torch.equal(dgamma, want[0]) and torch.equal(dbeta, want[1])
    dgamma, dbeta = start[0].clone(), start[1].clone()
    xt.xp_layernorm_backward(dy, x, None, mean, rstd, dx, dgamma, dbeta, work, accumulate=True)
    assert torch.equal(dgamma, want[0] + start[0]) and torch.equal(dbeta, want[1] + start[1])


@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("m_power", [-149, -130, -115, -100, -60, 0, 60, 110, 126])
def test_states_at_every_magnitude(xt, m_power, lead):
    # 8-bit states: weights, codes and scales of a step, in whole turns and at the end, are the fp32 program's, and so are
    # weights and states in fp32; subnormal numbers and blocks of zeros among them
    torch = torch_cuda()
    n, step, lr = 4096 + 77, 9, 1e-3
    half = np.full(n, 1 << 15)

    def dev(a):
        buf = torch.zeros(len(a) + lead, dtype=torch.from_numpy(a).dtype, device="cuda")
        buf[lead:] = torch.from_numpy(a)
        return buf[lead:]

    hashes = train.rounding_bits(77, step + 1, range(n))
    for v_power in (-149, -130, -120, -110, -95, -60, 0, 60, 110, 126):
        rng = np.random.default_rng(100000 + 200 * m_power + v_power)
        g = (rng.standard_normal(n) * 2.0 ** min(m_power - 2, 55) * (rng.random(n) < 0.7)).astype(np.float32)
        m = (np.clip(rng.standard_normal(n) * 2.0 ** (m_power + rng.integers(-12, 1, n)), -1.5e38, 1.5e38) * (rng.random(n) < 0.8)).astype(np.float32)
        v = (np.clip(rng.random(n) * 2.0 ** (v_power + rng.integers(-12, 1, n)), 0, 1.5e38) * (rng.random(n) < 0.9)).astype(np.float32)
        p = rng.standard_normal(n).astype(np.float32)
        (cm, sm), (cv, sv) = train.encode(m, half, True), train.encode(v, half, False)
        t = [dev(a) for a in (p, g, cm, cv, sm, sv)]
        m_out, v_out = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        xt.xp_state8_decode(t[2], t[4], t[3], t[5], m_out, v_out)
        m, v = train.decode(cm, sm, True).astype(np.float32), train.decode(cv, sv, False).astype(np.float32)
        assert np.array_equal(m_out.cpu().numpy(), m) and np.array_equal(v_out.cpu().numpy(), v)
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            want = train.adamw(p, g, m, v, step + 1, lr, 0.0)
        assert np.isfinite(want[1]).all() and np.isfinite(want[2]).all()
        group = xt.xp_group_create([t[0]], [t[1]], [t[2]], [t[3]], m_scales=[t[4]], v_scales=[t[5]], seed=77, step=step)
        xt.xp_adamw_step(group, lr)
        xt.xp_group_destroy(group)
        codes = [*train.encode(want[1], hashes[0], True), *train.encode(want[2], hashes[1], False)]
        for got, ref in zip((t[0], t[2], t[4], t[3], t[5]), (want[0], *codes)):
            assert np.array_equal(got.cpu().numpy(), ref), v_power
        t = [dev(a) for a in (p, g, m, v)]
        group = xt.xp_group_create([t[0]], [t[1]], [t[2]], [t[3]], step=step)
        xt.xp_adamw_step(group, lr)
        xt.xp_group_destroy(group)
        for got, ref in zip((t[0], t[2], t[3]), want):
            assert np.array_equal(got.cpu().numpy(), ref), v_power


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_every_code_under_every_scale(xt, out):
    torch = torch_cuda()
    codes, scales = np.tile(np.arange(256, dtype=np.uint8), 256), np.repeat(np.arange(256, dtype=np.uint8), 8)
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    got = [torch.empty(len(codes), dtype=_types(torch, out)[0], device="cuda") for _ in range(2)]
    xt.xp_state8_decode(c, s, c, s, *got)
    for values, signed in zip(got, (True, False)):
        with np.errstate(over="ignore"):
            want = train.decode(codes, scales, signed).astype(np.float32).astype(np.float64)
        assert np.array_equal(_f64(values), want, equal_nan=True)

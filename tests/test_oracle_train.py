"""The training operators' oracle and refusals, on the CPU: the layer norm gradient against differences, the 8-bit
states' rounding against its definition, the header against the binding, and every argument error that needs no GPU."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "xp_train.h")


@pytest.fixture(scope="module")
def xt():
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_train as xt
    return xt


# ---- formulas

@pytest.mark.parametrize("rows,cols,affine", [(3, 5, True), (1, 2, True), (4, 17, False)])
def test_layernorm_gradient_equals_differences(rows, cols, affine):
    # central differences of L = sum(dy * y) with step h: error about h^2 |L'''| / 6 + 2^-52 |L| / h; with h = 1e-5 and
    # values of order 1 to 100 both are below 1e-8
    rng = np.random.default_rng(cols)
    x, dy = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    gamma, beta = (1 + 0.3 * rng.standard_normal(cols), rng.standard_normal(cols)) if affine else (None, None)

    def loss(x, gamma, beta):
        return float((dy * train.layernorm_forward(x, gamma, beta, 1e-2)[0]).sum())

    _, mean, rstd = train.layernorm_forward(x, gamma, beta, 1e-2)
    dx, dgamma, dbeta = train.layernorm_backward(dy, x, gamma, mean, rstd)
    h = 1e-5
    checks = [(x, dx, 0)] + ([(gamma, dgamma, 1), (beta, dbeta, 2)] if affine else [])
    for value, grad, k in checks:
        for i in np.ndindex(value.shape):
            args = [[x, gamma, beta] for _ in range(2)]
            for a, s in zip(args, (h, -h)):
                a[k] = value.copy()
                a[k][i] += s
            num = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            assert abs(num - grad[i]) < 1e-7 * max(1, np.abs(grad).max())


def test_adamw_first_step_moves_by_lr():
    # at t = 1 with zero states m / (1 - b1) = g and v / (1 - b2) = g^2: the step is lr * sign(g), up to eps
    p, g = np.zeros(8), np.array([1e-3, -2.0, 5.0, 1e-1, -1e-2, 3.0, -4.0, 1.0])
    q, m, v = train.adamw(p, g, np.zeros(8), np.zeros(8), 1, 0.01, 0.1)
    assert np.allclose(q, -0.01 * np.sign(g), rtol=2e-5)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.001 * g * g)


def test_state8_codes_stand_for_their_values():
    # every code of a block whose scale is E decodes to (c + 8 E - K) << 20 read as fp32
    for signed, k in ((True, 119), (False, 247)):
        for e in (1, 40, 127, 254):
            codes = np.arange(256, dtype=np.uint8)
            got = train.decode(codes, np.full(8, e, np.uint8), signed)
            mag = codes.astype(np.int64) % 128 if signed else codes.astype(np.int64)
            bits = np.where(mag == 0, 0, np.maximum(mag + 8 * e - k, 0) << 20)
            want = bits.astype(np.uint32).view(np.float32).astype(np.float64)
            want = np.where(signed & (codes >= 128), -want, want)
            ok = (mag + 8 * e - k >= 0) | (mag == 0)
            ok &= bits < 0x7f800000      # the block's scale leaves no larger code
            assert np.array_equal(got[ok], want[ok])
    assert np.isnan(train.decode(np.zeros(32, np.uint8), np.array([255], np.uint8), False)).all()


@pytest.mark.parametrize("signed", [True, False])
def test_state8_rounding_keeps_the_mean(signed):
    # over all 65536 hashes a value's mean code value is the value itself, to within half a hash step (2^-17 of a code)
    rng = np.random.default_rng(3)
    x = np.zeros(32, np.float32)
    x[0], x[1] = 1.0, rng.uniform(0.01, 0.9)
    total = 0.0
    hs = np.arange(0, 65536, 16)
    for h in hs:
        c, s = train.encode(x, np.full(32, h), signed)
        total += train.decode(c, s, signed)[1]
    quantum = 2.0 ** (np.floor(np.log2(x[1])) - 3)
    assert abs(total / len(hs) - x[1]) <= 16 * quantum / 65536
    # codes are exact for values they stand for, whatever the hash
    c, s = train.encode(x, np.full(32, 65535), signed)
    y = train.decode(c, s, signed).astype(np.float32)
    for h in (0, 1, 40000, 65535):
        c2, s2 = train.encode(y, np.full(32, h), signed)
        assert np.array_equal(train.decode(c2, s2, signed).astype(np.float32), y)


def test_state8_extremes():
    x = np.float32([3e38, 1e-30, 1e-20, 0, 2e-38] + [0] * 27)
    c, s = train.encode(x, np.zeros(32, np.int64), False)
    d = train.decode(c, s, False)
    assert d[3] == 0 and (d[[0, 1, 2, 4]] > 0).all()       # a positive v stays positive
    c, s = train.encode(-x, np.zeros(32, np.int64), True)
    d = train.decode(c, s, True)
    assert d[0] < -2e38 and (d[1:] == 0).all() and (c[1:] == 0).all()
    c, s = train.encode(np.full(32, np.float32(np.finfo(np.float32).max)), np.full(32, 65535), False)
    assert s[0] == 254 and np.isinf(train.decode(c, s, False).astype(np.float32)).all()   # the next power is out of range


def test_rounding_bits_look_uniform():
    # 2^14 hashes: means of the 16-bit halves within 5 standard errors, steps and positions uncorrelated
    n = 1 << 14
    a, b = train.rounding_bits(7, 11, range(n))
    c, _ = train.rounding_bits(7, 12, range(n))
    for x in (a, b, c):
        assert abs(x.mean() / 65535 - 0.5) < 5 / np.sqrt(12 * n)
    for x, y in ((a, b), (a, c), (a[1:], a[:-1]), (b[32:], b[:-32])):
        assert abs(np.corrcoef(x[: len(y)], y)[0, 1]) < 5 / np.sqrt(n)
    hi, _ = train.rounding_bits(7, 11, [i + (1 << 32) for i in range(64)])
    assert (hi != a[:64]).sum() > 60


# ---- the boundary

def test_every_declared_symbol_is_exported(xt):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(xp_[a-z0-9_]+)\s*\(", src)))
    assert sorted(xt.EXPORTS) == names
    out = subprocess.run(["nm", "-D", "--defined-only", xt.xp.library_path()], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r"\bT (xp_[a-z0-9_]+)", out))


@pytest.mark.parametrize("name", ["xp_tensor", "xp_group_config", "xp_grad_report"])
def test_binding_mirrors_the_header(xt, name):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, src).group(1)
    fields = []
    for decl in body.split(";"):
        names = re.sub(r"\[\d+\]", "", decl).strip()
        if names:
            first, *rest = names.split(",")
            fields += [first.split()[-1].lstrip("*")] + [r.strip().lstrip("*") for r in rest]
    assert fields == [f for f, _ in getattr(xt, name)._fields_]


def test_constants(xt):
    src = open(HEADER).read()
    assert int(re.search(r"XP_LAYERNORM_MAX_COLS \(\(size_t\)(\d+)\)", src).group(1)) == xt.XP_LAYERNORM_MAX_COLS
    assert 1 << int(re.search(r"XP_LAYERNORM_MAX_ROWS \(\(size_t\)1 << (\d+)\)", src).group(1)) == xt.XP_LAYERNORM_MAX_ROWS
    assert int(re.search(r"XP_STATE8_BLOCK (\d+)", src).group(1)) == xt.XP_STATE8_BLOCK == train.BLOCK


A = 1 << 20   # an address that no call here dereferences: every one is refused before a launch


@pytest.mark.parametrize("change", [
    {"x": None}, {"y": None}, {"cols": 0}, {"cols": 131073}, {"rows": (1 << 28) + 1}, {"x_stride": 63}, {"y_stride": 10},
    {"x": A + 1}, {"y": A + 3}, {"gamma": A + 2}, {"mean": A + 1}, {"eps": -1.0}, {"eps": float("nan")}, {"dtype": 2},
    {"wdtype": 0}, {"y": A + 4}, {"y": A, "y_stride": 65}, {"x_stride": 1 << 41}])
def test_layernorm_forward_refuses(xt, change):
    a = dict(x=A, x_stride=64, gamma=A * 3, beta=A * 4, y=A * 2, y_stride=64, mean=A * 5, rstd=A * 6, rows=8, cols=64,
             eps=1e-5, dtype=xt.XP_F32, wdtype=xt.XP_F32, stream=None) | change
    assert xt._lib.xp_layernorm_forward(*a.values()) == 1
    assert xt.xp.xp_last_error()


@pytest.mark.parametrize("change", [
    {"dy": None}, {"x": None}, {"dx": None}, {"mean": None}, {"rstd": None}, {"dgamma": None}, {"dbeta": None}, {"cols": 0},
    {"cols": 131073}, {"dx": A}, {"dx": A * 2 + 8}, {"dx": A * 2, "dx_stride": 66}, {"dtype": 7}, {"wdtype": 1},
    {"dy": A * 2 + 2}, {"gamma": A + 1}, {"dgamma": A + 1}, {"work": None}, {"nbytes": 100}, {"work": A * 9 + 8}, {"dx_stride": 3}])
def test_layernorm_backward_refuses(xt, change):
    a = dict(dy=A * 2, dy_stride=64, x=A, x_stride=64, gamma=A * 3, mean=A * 4, rstd=A * 5, dx=A * 6, dx_stride=64, dgamma=A * 7,
             dbeta=A * 8, rows=100, cols=64, dtype=xt.XP_F32, wdtype=xt.XP_F32, accumulate=0, work=A * 9, nbytes=1 << 30,
             stream=None) | change
    assert xt._lib.xp_layernorm_backward(*a.values()) == 1


def test_no_rows_is_no_launch(xt):
    f32 = xt.XP_F32
    assert xt._lib.xp_layernorm_forward(None, 4, None, None, None, 4, None, None, 0, 4, 1e-5, f32, f32, None) == 0
    assert xt._lib.xp_layernorm_backward(None, 4, None, 4, None, None, None, None, 4, None, None, 0, 4, f32, f32, 0, None, 0, None) == 0
    assert xt.xp_layernorm_workspace(0, 100) == 0


def _create(xt, cfg=(), tensor=(), n=1):
    c = dict(beta1=0.9, beta2=0.99, eps=1e-8, param_dtype=xt.XP_F32, grad_dtype=xt.XP_F32, state_dtype=xt.XP_F32, seed=0, step=0) | dict(cfg)
    t = dict(param=A, grad=A * 2, m=A * 3, v=A * 4, count=10, weight_decay=0.1) | dict(tensor)
    table = (xt.xp_tensor * 2)(xt.xp_tensor(**t), xt.xp_tensor(param=A, grad=A * 2, m=A * 3, v=A * 4, m_scale=A * 5, v_scale=A * 6, count=3))
    out = ctypes.c_void_p()
    return xt._lib.xp_group_create(ctypes.byref(xt.xp_group_config(**c)), n, table, ctypes.byref(out))


@pytest.mark.parametrize("cfg,tensor,n", [
    ({"beta1": 1.0}, {}, 1), ({"beta2": -0.1}, {}, 1), ({"eps": 0.0}, {}, 1), ({"eps": 1e-60}, {}, 1), ({"eps": float("nan")}, {}, 1),
    ({"param_dtype": 2}, {}, 1), ({"grad_dtype": 0}, {}, 1), ({"state_dtype": 4}, {}, 1), ({}, {"grad": None}, 1), ({}, {"m": None}, 1),
    ({}, {"v": None}, 1), ({"state_dtype": 0}, {}, 1), ({}, {"param": A + 2}, 1), ({}, {"grad": A + 1}, 1), ({}, {"copy": A + 1}, 1),
    ({}, {"m": A + 2}, 1), ({}, {"weight_decay": float("inf")}, 1), ({}, {"reserved": 1}, 1), ({}, {"param": None}, 2), ({}, {}, 0),
    ({}, {"count": 1 << 49}, 1)])
def test_group_create_refuses(xt, cfg, tensor, n):
    assert _create(xt, cfg, tensor, n) == 1


def test_null_groups_and_decodes_are_refused(xt):
    L = xt._lib
    assert L.xp_group_destroy(None) == 0
    assert L.xp_grad_norm(None, 1.0, 0.0, 0, A, None) == 1
    assert L.xp_adamw_step(None, 0.1, None, 1.0, None, 0, None) == 1
    assert L.xp_group_set_grads(None, None, None) == 1
    assert L.xp_group_set_step(None, 1, None) == 1
    assert L.xp_group_get_step(None, None, None) == 1
    assert L.xp_state8_decode(A, A, A, A, 32, A, A, 0, None) == 1
    assert L.xp_state8_decode(A, None, A, A, 32, A, A, xt.XP_F32, None) == 1
    assert L.xp_state8_decode(A, A, A, A, 32, A + 1, None, xt.XP_F32, None) == 1
    assert L.xp_state8_decode(None, None, None, None, 0, None, None, xt.XP_F32, None) == 0
    assert L.xp_layernorm_workspace(1 << 29, 4, ctypes.byref(ctypes.c_size_t())) == 1


def test_binding_refuses_shapes_that_differ(xt):
    torch = pytest.importorskip("torch")
    x, y = torch.zeros(4, 8), torch.zeros(4, 9)
    with pytest.raises(ValueError):
        xt.xp_layernorm_forward(x, None, None, y)
    with pytest.raises(ValueError):
        xt.xp_layernorm_forward(x, torch.zeros(7), None, torch.zeros(4, 8))
    with pytest.raises(ValueError):
        xt.xp_layernorm_forward(x, None, None, torch.zeros(8, 4).t())
    with pytest.raises(ValueError):
        xt.xp_layernorm_forward(x, None, None, torch.zeros(4, 8).bfloat16())
    with pytest.raises(ValueError):
        xt.xp_layernorm_forward(x.double(), None, None, x.double())
    with pytest.raises(ValueError):
        xt.xp_layernorm_backward(x, x, None, torch.zeros(4), torch.zeros(3), torch.zeros(4, 8))
    with pytest.raises(ValueError):
        xt.xp_group_create([x], [torch.zeros(32)], [torch.zeros(31)], [torch.zeros(32)])
    with pytest.raises(ValueError):
        xt.xp_group_create([x], [x, x])

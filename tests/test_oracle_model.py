"""Pins of the formulas of the layer in 8 bits (oracle.model): codes against torch's type, scales against their
definition, gradients against differences; and the boundary of include/xp_model.h."""
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "xp_model.h")


def test_codes_are_the_types():
    torch = pytest.importorskip("torch")
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(model.code_values(), want, equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 20000), np.exp(rng.uniform(-12, 6.1, 20000)), (want[:126] + want[1:127]) / 2, -want[:127]])
    got = model.nearest_code(x.astype(np.float32).astype(np.float64))
    assert np.array_equal(got, torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scales_are_the_least_that_fit():
    tops = np.concatenate([448 * 2.0 ** np.arange(-120, 120), np.nextafter(448 * 2.0 ** np.arange(-120, 120), np.inf), np.exp(np.linspace(-80, 80, 999))])
    e = model.scale_of(tops).astype(int)
    assert (tops <= 448 * 2.0 ** (e - 127)).all() and (tops > 448 * 2.0 ** (e - 128)).all()
    assert model.scale_of([0.0, 1e-45, np.inf, np.nan]).tolist() == [0, 0, 255, 255]


@pytest.mark.parametrize("block_rows", [1, 128])
def test_encoding_is_off_by_half_a_step(block_rows):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((130, 300)) * np.exp(rng.standard_normal((130, 1)) * 3)
    codes, scales = model.encode(x, block_rows)
    assert scales.shape == (-(-130 // block_rows), 3)
    power = np.repeat(np.repeat(2.0 ** (scales.astype(int) - 127), block_rows, 0)[:130], 128, 1)[:, :300]
    # half of 2^-3 of the power of two, which is 2^-6 of the scale at least
    step = np.maximum(2.0 ** np.floor(np.log2(np.abs(x))), power * 2.0 ** -6) / 8
    assert (np.abs(model.decode(codes, scales, block_rows) - x) <= step / 2).all()
    # encoded values are kept (by other codes where the largest was rounded down to 448 of the next scale: 449 -> 2 * 224)
    values = model.decode(codes, scales, block_rows)
    assert (model.decode(*model.encode(values, block_rows), block_rows) == values).all()


def _differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


def test_rmsnorm_gradient_is_that_of_differences():
    rng = np.random.default_rng(3)
    h, gamma, w, d = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    rstd = model.rmsnorm_forward(h, gamma)[1]
    dx, dgamma = model.rmsnorm_backward(w, h, gamma, rstd, d)
    assert np.abs(dx - _differences(lambda x: (model.rmsnorm_forward(x, gamma)[0] * w + x * d).sum(), h)).max() < 1e-7
    assert np.abs(dgamma - _differences(lambda g: (model.rmsnorm_forward(h, g)[0] * w).sum(), gamma)).max() < 1e-7


@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_distillation_gradient_is_that_of_differences(temperature):
    rng = np.random.default_rng(4)
    z, t, d = rng.standard_normal((4, 9)) * 2, rng.standard_normal((4, 5)) * 2, rng.standard_normal(4)
    ids = np.array([[0, 3, 8, 2, 1], [4, 4, 4, 1, 1], [2, -1, 9, 7, -5], [-1, -1, 40, -1, -1]])   # one twice and more; some that name none
    loss, lse = model.distill_forward(z, ids, t, temperature)
    assert loss[3] == 0 and lse[3] == 0 and (loss[:3] > 0).all()
    got = model.distill_backward(z, ids, t, lse, d, temperature)
    want = _differences(lambda x: (model.distill_forward(x, ids, t, temperature)[0] * d).sum(), z)
    assert np.abs(got - want).max() < 1e-7 and (got[3] == 0).all()
    # one entry is the cross entropy of a label
    one = model.distill_forward(z, ids[:, :1], t[:, :1])[0]
    assert np.allclose(one[:3], [-np.log(np.exp(z[i]) / np.exp(z[i]).sum())[ids[i, 0]] for i in range(3)])


def test_a_masked_vocabulary_and_a_masked_teacher():
    z = np.array([[1.0, -np.inf, 2.0, -np.inf]])
    loss, lse = model.distill_forward(z, np.array([[0, 2, 1]]), np.array([[0.5, 0.25, -np.inf]]))
    assert np.isfinite(loss).all() and np.isclose(lse[0], np.log(np.e + np.e ** 2))
    assert model.distill_forward(z, np.array([[0, 2]]), np.full((1, 2), -np.inf))[0][0] == 0
    assert model.distill_forward(z, np.array([[1]]), np.zeros((1, 1)))[0][0] == np.inf


# ---- the boundary

@pytest.fixture(scope="module")
def xm():
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_model as xm
    return xm


def test_every_declared_symbol_is_exported(xm):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(xp_[a-z0-9_]+)\s*\(", src)))
    assert sorted(xm.EXPORTS) == names
    out = subprocess.run(["nm", "-D", "--defined-only", xm.xp.library_path()], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r"\bT (xp_[a-z0-9_]+)", out))


def test_limits_mirror_the_header(xm):
    found = dict(re.findall(r"#define (XP_[A-Z0-9_]+) \(?(?:\(size_t\))?(\d+(?: << \d+)?)\)?", open(HEADER).read()))
    assert {k: eval(v) for k, v in found.items()} == {k: getattr(xm, k) for k in (
        "XP_BLOCK8", "XP_MODEL_MAX_ROWS", "XP_MODEL_MAX_COLS", "XP_MODEL_MAX_STRIDE", "XP_DISTILL_MAX_TOP")}


def test_the_header_is_c(tmp_path):
    (tmp_path / "t.c").write_text('#include "xp_model.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", "-fsyntax-only",
                    str(tmp_path / "t.c")], check=True)

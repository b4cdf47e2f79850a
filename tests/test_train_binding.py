"""The training operators' host side, on the CPU: what the binding refuses before a call, against a library that records
its calls and launches nothing; the library's own rules, refusals and launches, against a runtime that runs nothing."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def fake(monkeypatch):
    """The binding over a library whose calls succeed and are recorded."""
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_train as xt

    class Library:
        def __init__(self):
            self.calls = []

        def xp_group_create(self, cfg, n, table, out):
            out._obj.value = 0x1000 + 16 * len(self.calls)
            return self.record("xp_group_create", n)

        def record(self, name, *args):
            self.calls.append((name, args))
            return 0

        def __getattr__(self, name):
            return lambda *args: self.record(name, *args)

    lib = Library()
    monkeypatch.setattr(xt, "_lib", lib)
    for alias, name in (("_norm", "xp_grad_norm"), ("_step", "xp_adamw_step"), ("_backward", "xp_layernorm_backward")):
        monkeypatch.setattr(xt, alias, getattr(lib, name))
    monkeypatch.setattr(xt, "lib", lib, raising=False)
    return xt


def _aligned(torch, n, dtype):
    """n elements that begin at a multiple of 16 bytes."""
    buf = torch.zeros(n + 16, dtype=dtype)
    return buf[-buf.data_ptr() % 16 // buf.element_size():][:n]


def test_other_gradients_have_the_groups_lengths_and_type(fake):
    torch = pytest.importorskip("torch")
    group = fake.xp_group_create(None, [torch.zeros(10), torch.zeros(2, 3), torch.zeros(0)])
    good = [torch.ones(10), torch.ones(3, 2), torch.ones(0)]
    made = len(fake.lib.calls)
    for bad in ([], good[:1], good[:2], good + [torch.ones(1)],                         # the library reads one pointer per tensor
                [torch.ones(9), *good[1:]], [torch.ones(11), *good[1:]],                # other lengths
                [good[0].bfloat16(), *good[1:]], [good[0].double(), *good[1:]],         # other types
                [good[0], torch.ones(2, 3).t(), good[2]], [torch.ones(20)[::2], *good[1:]]):   # not contiguous
        with pytest.raises(ValueError):
            fake.xp_group_set_grads(group, bad)
    assert len(fake.lib.calls) == made
    fake.xp_group_set_grads(group, good)
    name, (to, ptrs, _) = fake.lib.calls[-1]
    assert name == "xp_group_set_grads" and to == group and len(ptrs) == 3 and ptrs[0] == good[0].data_ptr() and ptrs[1] == good[1].data_ptr()
    fake.xp_group_destroy(group)
    with pytest.raises(ValueError):
        fake.xp_group_set_grads(group, good)
    assert fake.lib.calls[-1][0] == "xp_group_destroy"


def test_gradients_of_bf16_groups(fake):
    torch = pytest.importorskip("torch")
    group = fake.xp_group_create(None, [torch.zeros(10).bfloat16()])
    with pytest.raises(ValueError):
        fake.xp_group_set_grads(group, [torch.zeros(10)])
    fake.xp_group_set_grads(group, [torch.zeros(10).bfloat16()])
    fake.xp_group_destroy(group)


def test_reports_and_rates(fake):
    torch = pytest.importorskip("torch")
    assert ctypes.sizeof(fake.xp_grad_report) == 32
    good, none = _aligned(torch, 8, torch.float32), len(fake.lib.calls)
    for bad in (_aligned(torch, 7, torch.float32), _aligned(torch, 31, torch.uint8), _aligned(torch, 1, torch.float32).expand(8),
                _aligned(torch, 16, torch.float32)[::2]):
        with pytest.raises(ValueError):
            fake.xp_grad_norm(1, bad)
        with pytest.raises(ValueError):
            fake.xp_adamw_step(1, 0.1, report=bad)
    for bad in (torch.zeros(0), torch.zeros(1, dtype=torch.float64), torch.zeros(1, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            fake.xp_adamw_step(1, 0.1, lr_dev=bad)
    assert len(fake.lib.calls) == none
    fake.xp_grad_norm(1, good)
    fake.xp_grad_norm(1, _aligned(torch, 32, torch.uint8))
    fake.xp_adamw_step(1, 0.1, report=good, lr_dev=torch.zeros(3))
    assert [name for name, _ in fake.lib.calls[none:]] == ["xp_grad_norm", "xp_grad_norm", "xp_adamw_step"]


def test_workspaces(fake):
    torch = pytest.importorskip("torch")
    x, s = torch.zeros(4, 8), torch.zeros(4)
    with pytest.raises(ValueError):    # 4096 bytes by its shape, one in memory
        fake.xp_layernorm_backward(x, x, None, s, s, torch.zeros(4, 8), torch.zeros(8), torch.zeros(8), torch.zeros(1, dtype=torch.uint8).expand(4096))
    fake.xp_layernorm_backward(x, x, None, s, s, torch.zeros(4, 8), torch.zeros(8), torch.zeros(8), torch.zeros(4096, dtype=torch.uint8))
    assert fake.lib.calls[-1][0] == "xp_layernorm_backward"


@pytest.mark.parametrize("counts", ["[(1 << 40) + 1]", "[1 << 48]", "[1 << 40, 1]", "[1 << 39] * 300", "[1 << 40] * (1 << 20)"])
def test_a_group_of_too_many_elements_is_refused_before_its_tables(counts):
    # in a process of its own that may take 6 GiB: tables for them would be far larger
    code = f"""if True:
        import ctypes, re, resource, sys
        sys.path.insert(0, {ROOT!r})
        from collective_transport_plane_gb300 import xp_train as xt
        limit = int(re.search(r"XP_GROUP_MAX_ELEMENTS \\(\\(size_t\\)1 << (\\d+)\\)", open({ROOT!r} + "/include/xp_train.h").read()).group(1))
        assert xt.XP_GROUP_MAX_ELEMENTS == 1 << limit
        counts, A = {counts}, 1 << 20
        cfg = xt.xp_group_config(beta1=0.9, beta2=0.99, eps=1e-8, param_dtype=xt.XP_F32, grad_dtype=xt.XP_F32, state_dtype=xt.XP_F32)
        table = (xt.xp_tensor * len(counts))()
        for t, n in zip(table, counts):
            t.grad, t.count = A, n
        out = ctypes.c_void_p(77)
        resource.setrlimit(resource.RLIMIT_AS, (6 << 30, 6 << 30))
        status = xt._lib.xp_group_create(ctypes.byref(cfg), len(counts), table, ctypes.byref(out))
        print(status, out.value)"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert done.stdout.split() == ["1", "77"], (done.stdout, done.stderr[-500:])


@pytest.mark.parametrize("step", [(1 << 52) + 1, (1 << 64) - 1, -1])
def test_a_group_with_a_step_count_that_would_wrap_is_refused(step):
    # the bias corrections of step 2^64 would be those of step 0, infinite; -1 becomes 2^64 - 1 on its way
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_train as xt
    assert 1 << int(re.search(r"XP_GROUP_MAX_STEP \(\(uint64_t\)1 << (\d+)\)", open(os.path.join(ROOT, "include", "xp_train.h")).read()).group(1)) == xt.XP_GROUP_MAX_STEP
    cfg = xt.xp_group_config(beta1=0.9, beta2=0.99, eps=1e-8, param_dtype=xt.XP_F32, grad_dtype=xt.XP_F32, state_dtype=xt.XP_F32, step=step)
    table, out = (xt.xp_tensor * 1)(xt.xp_tensor(grad=1 << 20, count=5)), ctypes.c_void_p()
    assert xt._lib.xp_group_create(ctypes.byref(cfg), 1, table, ctypes.byref(out)) == xt.xp.XP_ERR_INVALID
    assert b"step" in xt._lib.xp_last_error()


@pytest.mark.parametrize("between", [0, 1, 39, 61, 99, 100, 101, 700, 739, -1, -39, -61, -100, -739])
def test_rows_that_share_bytes_are_refused(between):
    # 8 rows of 40 fp32, 100 apart: a second matrix shares bytes unless its rows lie whole in the 60 between
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_train as xt
    at, stride = 1 << 20, 100
    used = {r * stride + c for r in range(8) for c in range(40)}
    shared = any(r * stride + c + between in used for r in range(8) for c in range(40))
    assert shared
    if between != 0:     # x itself is allowed
        assert xt._lib.xp_layernorm_forward(at, stride, None, None, at + 4 * between, stride, None, None, 8, 40, 1e-5, xt.XP_F32, xt.XP_F32, None) == 1
        assert b"overlap" in xt._lib.xp_last_error()
    # dx never shares x
    assert xt._lib.xp_layernorm_backward(at * 2, stride, at, stride, None, at * 3, at * 4, at + 4 * between, stride, None, None, 8, 40,
                                         xt.XP_F32, xt.XP_F32, 0, None, 0, None) == 1
    assert b"overlap" in xt._lib.xp_last_error()


@pytest.fixture(scope="module")
def fake_runtime(tmp_path_factory):
    from collective_transport_plane_gb300 import build
    build.build()
    exe = str(tmp_path_factory.mktemp("fake") / "fake_runtime")
    objects = [os.path.join(build.BUILD, name) for name in ("xp_train.o", "xp_adamw.o", "xp_layernorm.o")]
    if not all(map(os.path.exists, objects)):
        build.build(force=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which(build.nvcc()))), "include")
    done = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", cuda, "-I", build.INCLUDE, os.path.join(ROOT, "tests", "fake_runtime.cpp"),
                           *objects, "-o", exe], capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    return lambda what: [[int(n) for n in line.split()] for line in subprocess.run([exe, what], capture_output=True, text=True, check=True).stdout.splitlines()]


def test_workspaces_are_the_current_devices(fake_runtime):
    # a part for each SM, and in clusters of two for each cluster that fits (here a quarter of the SMs)
    assert fake_runtime("devices") == [[152, 38], [76, 19], [10, 2], [76, 19], [152, 38]]


def test_threads_agree_on_a_workspace(fake_runtime):
    for _ in range(5):
        for got in fake_runtime("threads"):
            assert len(set(got)) == 1 and len(got) == 17 and got[0] > 0


def test_codes_below_the_least_pattern_stand_for_0():
    # codes of blocks of small scales whose patterns would be negative, and the code of pattern 0 that a v below 2^-129 takes
    import numpy as np

    from oracle import train
    for signed, k in ((True, 119), (False, 247)):
        for e in range(0, 40):
            codes = np.arange(128, dtype=np.uint8)
            got = train.decode(codes, np.full(4, e, np.uint8), signed)
            bits = np.where(codes == 0, 0, np.maximum(codes.astype(np.int64) + 8 * e - k, 0)) << 20
            assert np.array_equal(got, bits.astype(np.uint32).view(np.float32).astype(np.float64))
    c, e = train.encode(np.array([2.0 ** -140, 2.0 ** -129, 2.0 ** -100], np.float32), np.zeros(3, np.int64), False)
    assert c[0] == 247 - 8 * e[0].astype(int) and train.decode(c, e, False).tolist() == [0.0, 2.0 ** -129, 2.0 ** -100]


def test_every_launch_is_within_the_devices_limits(fake_runtime):
    # layer norm of 1 to 131072 columns in 1 to 2^20 rows, both types, aligned and not: dynamic shared memory, threads, CTAs
    # of a cluster, and CTAs that are no whole number of clusters
    (launches, smem, threads, cluster, broken), = fake_runtime("launches")
    assert launches > 100000 and smem <= 224 * 1024 and threads <= 1024 and cluster <= 8 and broken == 0

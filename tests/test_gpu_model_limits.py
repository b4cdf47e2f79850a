"""The operators of a layer in 8 bits at the limits of what their header promises: what a call waits for, and which
arguments equal calls may differ in."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def xm():
    torch_cuda()
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_model as xm
    return xm


def _ceil(a, b):
    return -(-a // b)


def _any_codes(torch, rows, cols, block_rows, seed):
    """Codes of every finite value and scales from 2^-7 to 2^6: sums of their products round."""
    gen = torch.Generator("cuda").manual_seed(seed)
    c = torch.randint(0, 127, (rows, cols), generator=gen, dtype=torch.uint8, device="cuda")
    c += 128 * torch.randint(0, 2, (rows, cols), generator=gen, dtype=torch.uint8, device="cuda")
    s = torch.randint(120, 134, (_ceil(rows, block_rows), _ceil(cols, 128)), generator=gen, dtype=torch.uint8, device="cuda")
    return c, s


def _apart(torch, t, step, offset=0):
    """The same bytes in rows a multiple of `step` apart, `offset` bytes into their buffer."""
    rows, cols = t.shape
    pitch = _ceil(cols, step) * step + (step if step < 128 and _ceil(cols, step) * step % 128 == 0 else 0)   # (below 128: off its multiples)
    m = torch.full((offset + rows * pitch,), 0x7F, dtype=torch.uint8, device="cuda")[offset:].view(rows, pitch)[:, :cols]
    m.copy_(t)
    return m


def test_the_status_call_waits_for_every_stream(xm):
    # a stream that does not wait for the legacy default stream, nor it for the stream
    torch = torch_cuda()
    a, sa = _any_codes(torch, 4096, 4096, 1, 1)
    b, sb = _any_codes(torch, 4096, 4096, 1, 2)
    c = torch.empty(4096, 4096, device="cuda")
    xm.xp_matmul8(a, sa, b, sb, c)
    torch.cuda.synchronize()
    st, behind = torch.cuda.Stream(), torch.cuda.Event()
    for _ in range(1000):
        xm.xp_matmul8(a, sa, b, sb, c, stream=st)
    behind.record(st)
    assert not behind.query()     # what the call is to wait for
    assert xm.xp_matmul8_status() == xm.XP_OK
    assert behind.query()
    torch.cuda.synchronize()


# Sizes of which one layout alone would be cut into parts of the columns differently than the other alone (with 152 SMs), and
# of tiles by one CTA, by CTAs that share one and by pairs.
@pytest.mark.parametrize("m,n,k", [(48, 1024, 4096), (192, 2048, 4096), (67, 511, 1588), (1, 2386, 1653), (391, 66, 6662), (762, 2152, 15524), (116, 9425, 10888),
                                   (2024, 435, 11067), (620, 3028, 12890), (1, 4096, 4096), (3000, 2000, 1000), (200, 300, 128)])
def test_equal_products_give_equal_bits_in_any_layout(xm, m, n, k):
    torch = torch_cuda()
    a, sa = _any_codes(torch, m, k, 1, m)
    b, sb = _any_codes(torch, n, k, 1, n)
    sa, sb = _apart(torch, sa, 4), _apart(torch, sb, 4)
    want = None
    for step_a, off_a, step_b, off_b in ((128, 0, 128, 0), (16, 0, 16, 0), (128, 0, 16, 0), (16, 0, 128, 0), (128, 16, 128, 64)):
        c = torch.empty(m, n, device="cuda")
        xm.xp_matmul8(_apart(torch, a, step_a, off_a), sa, _apart(torch, b, step_b, off_b), sb, c)
        want = c if want is None else want
        assert torch.equal(c, want), (step_a, off_a, step_b, off_b, int((c != want).sum()))


@pytest.mark.parametrize("m,n,k", [(1, 5, 128), (1, 128, 100), (3, 200, 300), (2, 129, 640), (300, 1000, 900), (600, 3000, 1300)])
def test_scales_of_exactly_their_size(xm, m, n, k):
    # rows of scales a multiple of four apart, the last one ending with its buffer; NaN scales behind every row and the buffer
    torch = torch_cuda()
    a, sa = _any_codes(torch, m, k, 1, m)
    b, sb = _any_codes(torch, n, k, 128, n)

    def exact(s):
        rows, cols = s.shape
        pitch = _ceil(cols, 4) * 4
        buf = torch.full(((rows - 1) * pitch + cols + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        view = torch.as_strided(buf, (rows, cols), (pitch, 1))
        view.copy_(s)
        return view

    a, b = _apart(torch, a, 16), _apart(torch, b, 16)
    c, want = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    xm.xp_matmul8(a, exact(sa), b, exact(sb), c, b_block_rows=128)
    xm.xp_matmul8(a, _apart(torch, sa, 4), b, _apart(torch, sb, 4), want, b_block_rows=128)
    assert torch.equal(c, want) and torch.isfinite(c).all()


# One CTA for a tile (one tile each, and several), CTAs that share a tile, pairs (one chunk of 4096 columns, and four).
GIVEN_UP = {"alone": (9000, 300, 16384), "alone, tile after tile": (20000, 600, 8192), "shared": (762, 2152, 15524), "pairs": (4096, 4096, 4096),
            "pairs, chunk after chunk": (2000, 4096, 16384)}


@pytest.mark.parametrize("form", list(GIVEN_UP))
def test_waits_that_are_given_up(xm, form):
    # With a limit of 1 us every warp that waits for a tile's first sums, 10 us and more of copies and products, gives up after a
    # try or two (4 us each), and all others in their turn.  C is NaN, the status says so, and copies, products and TMEM are
    # left in order: the next call with the usual limit is right, and so is one of another form.  In a process of its own,
    # whose status stays what it is.
    code = """
import sys
sys.path.insert(0, %r)
import torch
from collective_transport_plane_gb300 import xp, xp_model as xm
from tests.test_gpu_model_limits import GIVEN_UP, _any_codes
calls = []
for m, n, k in (GIVEN_UP[%r], (1, 4096, 4096)):
    (a, sa), (b, sb) = _any_codes(torch, m, k, 1, m), _any_codes(torch, n, k, 128, n)
    pitch = -(-k // 16) * 16
    a, b = (torch.nn.functional.pad(t, (0, pitch - k))[:, :k] for t in (a, b))
    sa, sb = (torch.nn.functional.pad(t, (0, -t.shape[1] %% 4))[:, :t.shape[1]] for t in (sa, sb))
    calls.append((a, sa, b, sb, torch.zeros(m, n, device="cuda")))
want = []
for call in calls:
    xm.xp_matmul8(*call, b_block_rows=128)
    want.append(call[-1].clone())
assert xm.xp_matmul8_status() == xm.XP_OK
for _ in range(3):
    for c in calls:
        c[-1].zero_()
    xp.xp_set_spin_timeout_ns(1000)
    xm.xp_matmul8(*calls[0], b_block_rows=128)
    assert xm.xp_matmul8_status() == xp.XP_ERR_TIMEOUT
    assert torch.isnan(calls[0][-1]).all(), int(torch.isnan(calls[0][-1]).sum())
    xp.xp_set_spin_timeout_ns(2_000_000_000)
    for call, w in zip(calls, want):
        xm.xp_matmul8(*call, b_block_rows=128)
        torch.cuda.synchronize()
        assert torch.equal(call[-1], w)
    xm.xp_matmul8(*calls[0], b_block_rows=128, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(calls[0][-1], want[0] + want[0])
print("in order")
""" % (ROOT, form)
    torch_cuda()
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0 and done.stdout.strip().endswith("in order"), done.stdout + done.stderr[-2000:]


@pytest.mark.parametrize("temperature", [0.5, 0.7, 1.0, 2.0])
@pytest.mark.parametrize("top,vocab", [(1, 50), (3, 50), (37, 3000)])
def test_a_teacher_whose_entries_are_all_masked_alike(xm, temperature, top, vocab):
    # logits that are all the type's lowest value say as much as logits that are all 0; one among others has no share
    torch = torch_cuda()
    z = torch.randn(4, vocab, generator=torch.Generator("cuda").manual_seed(top), device="cuda")
    ids = torch.arange(top, dtype=torch.int32, device="cuda").expand(4, top).contiguous()
    out = []
    for value in (torch.finfo(torch.float32).min, 0.0):
        t = torch.full((4, top), value, device="cuda")
        t[3, 0] = 1.0
        if value == 0.0:
            t[3, 1:] = -float("inf")
        loss, lse, d, g = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.ones(4, device="cuda"), torch.empty_like(z)
        xm.xp_distill_forward(z, ids, t, loss, lse, temperature)
        xm.xp_distill_backward(z, ids, t, lse, d, g, temperature)
        out.append((loss, lse, g))
    for masked, plain in zip(*out):
        assert torch.isfinite(plain).all() and torch.equal(masked, plain)


@pytest.mark.parametrize("m,n,k", [(33, 32000, 512), (3, 128256, 260), (200, 160001, 128), (130, 300, 32000), (70, 256, 128256), (2, 200, 160001), (5, 130, 1 << 20)])
def test_products_of_a_vocabulary(xm, m, n, k):
    # a last layer's logits and their gradient.  Products are multiples of 1/4 of 4 at most, and a million of them below 2^24
    # quarters: exact in any order
    from tests.test_gpu_model import _values, _whole
    torch = torch_cuda()
    a, sa = _whole(torch, m, k, 1, m, 126, 128)
    b, sb = _whole(torch, n, k, 128, n, 126, 128)
    want = (_values(torch, a, sa, 1) @ _values(torch, b, sb, 128).t()).float()
    c = torch.full((m, n), float("nan"), device="cuda")
    xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128)
    assert torch.equal(c, want)
    xm.xp_matmul8(a, sa, b, sb, c, b_block_rows=128, accumulate=True)
    assert torch.equal(c, 2 * want)

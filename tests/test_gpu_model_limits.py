"""The operators of a layer in 8 bits at the limits of what their header promises: what a call waits for, and which
arguments equal calls may differ in."""
import pytest

from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


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

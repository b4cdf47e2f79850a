"""The types of 8-bit matrices at the binding, on the CPU: codes are bytes or e4m3, scales bytes or e8m0, and neither passes as
the other."""
import pytest

from tests.test_model_binding import OnDevice, xm  # noqa: F401

torch = pytest.importorskip("torch")
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _bytes(rows, cols, dtype=torch.uint8):
    return OnDevice(torch.zeros(rows, cols, dtype=torch.uint8).view(dtype))


def _calls(xm, codes, scales):  # noqa: F811
    """One call of each kind with codes and scales of these types (300 x 200, blocks of one row)."""
    f = lambda *shape: OnDevice(torch.zeros(*shape))  # noqa: E731
    c, s, ct, st = _bytes(300, 200, codes), _bytes(300, 2, scales), _bytes(200, 300, codes), _bytes(200, 3, scales)
    return [lambda: xm.xp_block8_encode(f(300, 200), c, s), lambda: xm.xp_block8_encode(f(300, 200), codes_t=ct, scales_t=st),
            lambda: xm.xp_block8_decode(c, s, f(300, 200)), lambda: xm.xp_matmul8(c, s, _bytes(300, 200), _bytes(300, 2), f(300, 300)),
            lambda: xm.xp_matmul8(_bytes(300, 200), _bytes(300, 2), c, s, f(300, 300)), lambda: xm.xp_rmsnorm_forward(f(300, 200), None, y8=c, y8_scales=s)]


@pytest.mark.parametrize("codes", [torch.uint8, E4M3])
@pytest.mark.parametrize("scales", [torch.uint8, E8M0])
def test_their_own_types_and_bytes_are_taken(xm, codes, scales):  # noqa: F811
    for call in _calls(xm, codes, scales):
        call()
    assert len(xm.calls) == 6


@pytest.mark.parametrize("codes,scales", [(E8M0, torch.uint8), (E8M0, E8M0), (torch.uint8, E4M3), (E4M3, E4M3), (E8M0, E4M3), (torch.int8, torch.uint8),
                                          (torch.uint8, torch.int8), (torch.float8_e5m2, torch.uint8)])
def test_others_are_refused(xm, codes, scales):  # noqa: F811
    for call in _calls(xm, codes, scales):
        with pytest.raises(ValueError):
            call()
    assert xm.calls == []


def test_numbers_in_8_bits_are_no_floats(xm):  # noqa: F811
    for dtype in (torch.uint8, E4M3, E8M0):
        with pytest.raises(ValueError):
            xm.xp_block8_encode(_bytes(300, 200, dtype), _bytes(300, 200), _bytes(300, 2))
        with pytest.raises(ValueError):
            xm.xp_rmsnorm_forward(_bytes(300, 200, dtype), None)
    assert xm.calls == []

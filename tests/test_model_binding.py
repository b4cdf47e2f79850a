"""What the operators of the layer in 8 bits refuse, on the CPU: the binding before a call, over a library that records
its calls; the library before a launch, with addresses that nothing reads."""
import pytest

A = 1 << 20      # an address


class OnDevice:
    """A tensor as if on a device."""

    def __init__(self, t, device=0):
        self.t, self.device = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device


@pytest.fixture
def xm(monkeypatch):
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_model as xm
    xm.calls = []
    for alias in ("_encode", "_decode", "_matmul", "_forward", "_backward", "_distill", "_distill_back"):
        monkeypatch.setattr(xm, alias, lambda *args, name=alias: xm.calls.append((name, args)) or 0)
    monkeypatch.setattr(xm, "_device_of", lambda t: 0)
    return xm


@pytest.fixture
def lib():
    from collective_transport_plane_gb300 import build
    build.build()
    import collective_transport_plane_gb300.xp_model as xm
    return xm._lib


def _tensors():
    torch = pytest.importorskip("torch")
    f, u = torch.float32, torch.uint8
    on = lambda *shape, dtype=f: OnDevice(torch.zeros(*shape, dtype=dtype))  # noqa: E731
    return torch, on, f, u


def test_a_norm_and_its_arguments(xm):
    torch, on, f, u = _tensors()
    x, g, y8, s8 = on(6, 200), on(200), on(6, 200, dtype=u), on(6, 2, dtype=u)
    xm.xp_rmsnorm_forward(x, g, on(6, 200), on(6, 200), on(6, 200), on(6), y8, s8)
    xm.xp_rmsnorm_forward(x, None, None, rstd=on(6))
    assert len(xm.calls) == 2
    bad = [dict(y=on(6, 201)), dict(y=on(6, 200, dtype=torch.bfloat16)), dict(gamma=on(199)), dict(gamma=on(200, dtype=u)), dict(rstd=on(5)),
           dict(rstd=on(6, dtype=torch.bfloat16)), dict(y8=y8), dict(y8_scales=s8), dict(y8=y8, y8_scales=on(6, 3, dtype=u)),
           dict(y8=on(6, 200), y8_scales=s8), dict(residual=on(5, 200), added=x), dict(y=OnDevice(torch.zeros(200, 6).t())),
           dict(y=OnDevice(torch.zeros(6, 200), 1)), dict(y=OnDevice(torch.zeros(6, 200), -1)), dict(x=on(6, 200, dtype=u)),
           dict(x=OnDevice(torch.zeros(6, 200, dtype=torch.float64)))]
    for change in bad:
        with pytest.raises(ValueError):
            xm.xp_rmsnorm_forward(**({"x": x, "gamma": g, "y": on(6, 200)} | change))
    assert len(xm.calls) == 2
    back = dict(dy=x, h=x, gamma=g, rstd=on(6), dx=x, dgamma=on(200), workspace=on(4096))
    xm.xp_rmsnorm_backward(**back)
    for change in (dict(dy=on(6, 199)), dict(dx=on(7, 200)), dict(dadded=on(6, 200, dtype=torch.bfloat16)), dict(dgamma=on(6)), dict(rstd=on(200)),
                   dict(dgamma=on(200, dtype=torch.bfloat16)), dict(workspace=OnDevice(torch.zeros(1, dtype=u).expand(4096))),
                   dict(workspace=OnDevice(torch.zeros(4096), -1))):
        with pytest.raises(ValueError):
            xm.xp_rmsnorm_backward(**(back | change))
    assert len(xm.calls) == 3


def test_matrices_in_8_bits(xm):
    torch, on, f, u = _tensors()
    x, c, s, ct, st = on(300, 200), on(300, 200, dtype=u), on(300, 2, dtype=u), on(200, 300, dtype=u), on(200, 3, dtype=u)
    xm.xp_block8_encode(x, c, s, ct, st)
    xm.xp_block8_encode(x, c, on(3, 2, dtype=u), block_rows=128)
    xm.xp_block8_encode(x, codes_t=ct, scales_t=st)
    xm.xp_block8_encode(x, OnDevice(c.t.view(torch.float8_e4m3fn)), s)
    xm.xp_block8_decode(c, s, x)
    assert [name for name, _ in xm.calls] == ["_encode"] * 4 + ["_decode"]
    for args, kw in (((x, c, on(3, 2, dtype=u)), {}), ((x, c, s), dict(block_rows=128)), ((x, c, s), dict(block_rows=64)), ((x, c), {}), ((x, ct, st), {}),
                     ((x, None, None, c, s), {}), ((c, c, s), {}), ((x, on(300, 200), s), {})):
        with pytest.raises(ValueError):
            xm.xp_block8_encode(*args, **kw)
    for args in ((c, s, on(300, 201)), (c, s, c), (c, on(300, 1, dtype=u), x), (None, None, x)[:0] or (c, None, x)):
        with pytest.raises(ValueError):
            xm.xp_block8_decode(*args)
    a, sa, b, sb, out = on(6, 200, dtype=u), on(6, 2, dtype=u), on(300, 200, dtype=u), on(3, 2, dtype=u), on(6, 300)
    n = len(xm.calls)
    xm.xp_matmul8(a, sa, b, sb, out, b_block_rows=128)
    xm.xp_matmul8(a, sa, c, s, out, accumulate=True)
    for args, kw in (((a, sa, b, sb, out), {}), ((a, sa, b, sb, on(300, 6)), dict(b_block_rows=128)), ((a, sa, on(300, 201, dtype=u), sb, out), dict(b_block_rows=128)),
                     ((a, sb, b, sb, out), dict(b_block_rows=128)), ((a, sa, b, sb, on(6, 300, dtype=u)), dict(b_block_rows=128)),
                     ((a, sa, b, sb, out), dict(b_block_rows=128, a_block_rows=2)), ((on(6, 200), sa, b, sb, out), dict(b_block_rows=128))):
        with pytest.raises(ValueError):
            xm.xp_matmul8(*args, **kw)
    assert len(xm.calls) == n + 2


def test_distillation(xm):
    torch, on, f, u = _tensors()
    z, ids, t, loss = on(6, 50), on(6, 4, dtype=torch.int32), on(6, 4), on(6)
    xm.xp_distill_forward(z, ids, t, loss, on(6), 2.0)
    xm.xp_distill_forward(z, ids, t, loss)
    xm.xp_distill_backward(z, ids, t, on(6), on(6), z)
    for args in ((z, on(6, 4, dtype=torch.int64), t, loss), (z, on(5, 4, dtype=torch.int32), on(5, 4), loss), (z, ids, on(6, 3), loss), (z, ids, t, on(5)),
                 (z, ids, on(6, 4, dtype=torch.bfloat16), loss), (z, ids, t, loss, on(7)), (on(6, 50, dtype=u), ids, t, loss),
                 (z, OnDevice(torch.zeros(6, 8, dtype=torch.int32)[:, ::2]), t, loss), (z, OnDevice(ids.t, -1), t, loss)):
        with pytest.raises(ValueError):
            xm.xp_distill_forward(*args)
    for args in ((z, ids, t, on(6), on(6), on(6, 51)), (z, ids, t, on(6), on(6), on(6, 50, dtype=torch.bfloat16)), (z, ids, t, on(5), on(6), z)):
        with pytest.raises(ValueError):
            xm.xp_distill_backward(*args)
    assert len(xm.calls) == 3


def _refused(lib, name, good, changes):
    """Every change of one argument of a call that would be made is refused by the library."""
    for at, value, word in changes:
        args = list(good)
        args[at] = value
        assert getattr(lib, name)(*args) == 1, (name, at, value)
        assert word.encode() in lib.xp_last_error(), (name, at, value, lib.xp_last_error())


F32, BF16, U8 = 3, 4, 0


def test_the_library_refuses_encodings(lib):
    #       x  stride rows cols type rows128 codes stride scales stride codes_t stride scales_t stride stream
    good = [A, 256, 200, 256, F32, 1, 2 * A, 256, 3 * A, 2, 4 * A, 208, 5 * A, 2, None]
    _refused(lib, "xp_block8_encode", good, [
        (0, None, "x is NULL"), (0, A + 2, "aligned"), (1, 255, "apart overlap"), (1, (1 << 36) + 4, "apart"), (2, (1 << 28) + 1, "rows"), (3, (1 << 20) + 1, "cols"),
        (4, U8, "dtype"), (5, 2, "block_rows"), (7, 255, "codes"), (8, None, "scales is NULL"), (9, 1, "scales"), (11, 199, "codes_t"), (12, None, "NULL"),
        (6, A + 1000, "overlap"), (8, 2 * A + 128, "overlap"), (10, 2 * A, "overlap"), (12, 3 * A + 1, "overlap"), (2, (1 << 20) + 1, "transposed")])
    both = list(good)
    both[6] = both[10] = None
    assert lib.xp_block8_encode(*both) == 1 and b"codes and codes_t" in lib.xp_last_error()
    empty = list(good)
    empty[0], empty[2] = None, 0
    assert lib.xp_block8_encode(*empty) == 0
    good = [A, 256, 2 * A, 2, 200, 256, 1, 3 * A, 256, F32, None]
    _refused(lib, "xp_block8_decode", good, [(0, None, "NULL"), (2, None, "NULL"), (7, None, "NULL"), (6, 7, "block_rows"), (7, A + 512, "overlap"), (7, 3 * A + 2, "aligned"),
                                             (9, U8, "dtype"), (8, 255, "overlap")])


def test_the_library_refuses_products(lib):
    #       a stride scales stride rows128 b stride scales stride rows128 c stride m n k type accumulate stream
    good = [A, 256, 2 * A, 4, 1, 3 * A, 256, 4 * A, 4, 128, 5 * A, 300, 64, 300, 256, F32, 0, None]
    _refused(lib, "xp_matmul8", good, [
        (0, None, "a is NULL"), (2, None, "scales is NULL"), (5, None, "b is NULL"), (7, None, "NULL"), (10, None, "c is NULL"), (0, A + 8, "16 bytes"), (1, 264, "16 bytes"),
        (5, 3 * A + 4, "16 bytes"), (6, 255, "overlap"), (2, 2 * A + 2, "4 bytes"), (3, 6, "4 bytes"), (7, 4 * A + 1, "4 bytes"), (4, 3, "block_rows"), (9, 0, "block_rows"),
        (10, 5 * A + 2, "aligned"), (11, 299, "overlap"), (15, U8, "dtype"), (10, A + 64, "overlaps"), (10, 4 * A, "overlaps"), (12, (1 << 28) + 1, "rows"),
        (13, (1 << 28) + 1, "rows"), (14, (1 << 20) + 1, "cols")])
    add = list(good)
    add[15], add[16] = BF16, 1
    assert lib.xp_matmul8(*add) == 1 and b"added" in lib.xp_last_error()
    for at in (12, 13):    # nothing to compute
        empty = [None, 0, None, 0, 1, None, 0, None, 0, 1, None, 0, 5, 5, 5, F32, 0, None]
        empty[at] = 0
        assert lib.xp_matmul8(*empty) == 0
    keep = list(good)
    keep[14], keep[16] = 0, 1
    assert lib.xp_matmul8(*keep) == 0    # c + nothing


def test_the_library_refuses_norms(lib):
    #       x stride residual stride gamma added stride y stride y8 stride scales stride rstd rows cols eps type wtype stream
    good = [A, 128, 2 * A, 128, 3 * A, 4 * A, 128, 5 * A, 128, 6 * A, 128, 7 * A, 1, 8 * A, 50, 128, 1e-5, F32, F32, None]
    _refused(lib, "xp_rmsnorm_forward", good, [
        (0, None, "x is NULL"), (5, None, "together"), (2, None, "together"), (4, 3 * A + 2, "aligned"), (13, 8 * A + 2, "aligned"), (1, 127, "overlap"), (15, 0, "cols is 0"),
        (16, -1.0, "eps"), (16, float("nan"), "eps"), (16, float("inf"), "eps"), (17, U8, "dtype"), (18, U8, "dtype"), (11, None, "NULL"), (5, A + 4, "overlaps"),
        (7, 4 * A, "overlap"), (9, A, "overlaps"), (13, A, "overlaps"), (7, 3 * A, "overlaps"), (14, (1 << 28) + 1, "rows"), (15, (1 << 20) + 1, "cols")])
    #       dy stride h stride gamma rstd dadded stride dx stride dgamma rows cols type wtype accumulate workspace bytes stream
    good = [A, 128, 2 * A, 128, 3 * A, 4 * A, 5 * A, 128, 6 * A, 128, 7 * A, 50, 128, F32, F32, 0, 8 * A, 1 << 20, None]
    _refused(lib, "xp_rmsnorm_backward", good, [
        (0, None, "NULL"), (2, None, "NULL"), (5, None, "rstd is NULL"), (8, None, "NULL"), (16, None, "workspace"), (16, 8 * A + 8, "workspace"), (17, 100, "needed"),
        (8, 2 * A, "overlaps"), (8, A + 4, "overlaps"), (10, 2 * A, "overlaps"), (16, 6 * A, "overlap"), (10, 7 * A + 1, "aligned"), (13, U8, "dtype"), (12, 0, "cols")])
    assert lib.xp_rmsnorm_workspace(5, 5, None) == 1


def test_the_library_refuses_distillations(lib):
    #       z stride ids teacher rows vocab top T loss lse type stream
    good = [A, 1000, 2 * A, 3 * A, 20, 1000, 8, 1.0, 4 * A, 5 * A, F32, None]
    nan = float("nan")
    both = [(0, None, "NULL"), (2, None, "NULL"), (3, None, "NULL"), (2, 2 * A + 1, "aligned"), (1, 999, "overlap"), (4, (1 << 28) + 1, "rows"), (5, 0, "vocab"),
            (5, (1 << 20) + 1, "cols"), (6, 1025, "top")]
    _refused(lib, "xp_distill_forward", good, both + [(7, v, "temperature") for v in (0.0, -1.0, nan, float("inf"), 1e-7, 1e7)] + [
        (8, None, "loss"), (8, 4 * A + 1, "loss"), (9, 5 * A + 2, "lse"), (10, U8, "dtype"), (8, A, "overlaps"), (9, 4 * A + 4, "overlaps"), (8, 2 * A, "overlaps")])
    #       z stride ids teacher lse dloss rows vocab top T dlogits stride type stream
    good = [A, 1000, 2 * A, 3 * A, 4 * A, 5 * A, 20, 1000, 8, 1.0, 6 * A, 1000, F32, None]
    _refused(lib, "xp_distill_backward", good, [(0, None, "NULL"), (4, None, "NULL"), (5, None, "NULL"), (10, None, "NULL"), (10, A + 4, "overlaps"), (10, 2 * A, "overlaps"),
                                                (10, 5 * A, "overlaps"), (11, 999, "overlap"), (9, nan, "temperature"), (12, U8, "dtype")])

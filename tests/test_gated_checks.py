"""CPU checks of the gated and 4-bit matrix-vector operators' refusals: the C ABI
rejects invalid calls on the host, the binding rejects tensors of another size, type or
layout.  Nothing reaches a GPU."""
import ctypes

import pytest
import torch

P, I = ctypes.c_void_p, ctypes.c_int


@pytest.fixture(scope="module")
def lib():
    from fine_grained_fp8_persistent_gb300 import build
    return ctypes.CDLL(build.build())


def _err(lib):
    lib.fgf8_last_error.restype = ctypes.c_char_p
    return lib.fgf8_last_error().decode()


AL, MIS = P(0x10000), P(0x10008)     # never dereferenced: every call below is refused first


def test_gated_f16_refusals(lib):
    f = lib.gated_f16
    f.argtypes = [P] * 6 + [I] * 5 + [P]
    ok = [AL] * 4 + [None, None]
    assert f(*ok, -1, 16, 16, 0, 0, None) == 1
    assert f(*ok, 4, 0, 16, 0, 0, None) == 1
    assert f(*ok, 4, 16, 16, 2, 0, None) == 1 and "dtype" in _err(lib)
    assert f(*ok, 4, 16, 16, 0, 2, None) == 1 and "activation" in _err(lib)
    assert f(*ok, 4, 12, 16, 0, 0, None) == 2 and "multiples of 8" in _err(lib)
    assert f(*ok, 4, 16, 20, 0, 0, None) == 2
    assert f(AL, None, AL, AL, None, None, 4, 16, 16, 0, 0, None) == 1
    assert f(AL, AL, AL, AL, AL, None, 4, 16, 16, 0, 0, None) == 1 and "together" in _err(lib)
    assert f(AL, AL, MIS, AL, None, None, 4, 16, 16, 0, 0, None) == 3
    assert f(None, None, None, None, None, None, 0, 16, 16, 1, 1, None) == 0      # no tokens: a no-op


def test_gated_f16_backward_refusals(lib):
    f = lib.gated_f16_backward
    f.argtypes = [P] * 10 + [I] * 5 + [P]
    ok = [AL] * 10
    assert f(*ok, -1, 16, 16, 0, 0, None) == 1
    assert f(*ok, 4, 16, 0, 0, 0, None) == 1
    assert f(*ok, 4, 16, 16, 0, -1, None) == 1
    assert f(*ok, 4, 16, 4, 0, 0, None) == 2
    assert f(*ok[:8], None, AL, 4, 16, 16, 0, 0, None) == 1
    assert f(*ok[:2], MIS, *ok[3:], 4, 16, 16, 0, 0, None) == 3
    ws = lib.fgf8_gated_backward_ws_bytes
    ws.restype = ctypes.c_longlong
    assert ws(0, 16) == 0 and ws(5, 16) >= 2 * 2 * 5 * 16
    assert ws(1 << 20, 1 << 14) >= 4 << 34                                       # past 32 bits
    assert ws(-1, 16) == -1 and ws(4, 0) == -1 and ws(4, 12) == -1


@pytest.mark.parametrize("gated", [False, True])
def test_gemv_fp4_refusals(lib, gated):
    if gated:
        lib.gated_gemv_fp4.argtypes = [P] * 6 + [I] * 6 + [P]

        def f(ptrs, M, N, K, fmt, dtype, act=0):
            return lib.gated_gemv_fp4(*ptrs[:3], *ptrs[1:3], ptrs[3], M, N, K, fmt, dtype, act, None)
    else:
        lib.gemv_fp4.argtypes = [P] * 4 + [I] * 5 + [P]

        def f(ptrs, M, N, K, fmt, dtype):
            return lib.gemv_fp4(*ptrs, M, N, K, fmt, dtype, None)
    ok = [AL] * 4
    assert f(ok, -1, 16, 64, 0, 0) == 1
    assert f(ok, 1, 0, 64, 0, 0) == 1
    assert f(ok, 1, 16, 64, 2, 0) == 1 and "format" in _err(lib)
    assert f(ok, 1, 16, 64, 0, 3) == 1 and "dtype" in _err(lib)
    assert f(ok, 1, 16, 96, 0, 0) == 2 and "multiple of 64" in _err(lib)
    assert f(ok, 17, 16, 64, 0, 0) == 2 and "16 rows" in _err(lib)
    assert f([AL, AL, None, AL], 1, 16, 64, 0, 0) == 1
    assert f([MIS, AL, AL, AL], 1, 16, 64, 1, 1) == 3
    assert f([None] * 4, 0, 16, 64, 1, 1) == 0
    if gated:
        assert f(ok, 1, 16, 64, 0, 0, act=5) == 1


# ----------------------------------------------------------------- the binding
class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            self.calls.append(name)
            return 0
        return f


@pytest.fixture()
def fg(monkeypatch):
    from fine_grained_fp8_persistent_gb300 import binding
    rec = _Recorder()
    monkeypatch.setattr(binding, "_launch", lambda name, stream, tensors, ints: rec.calls.append(name))
    binding.recorder = rec
    return binding


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_gated(fg):
    x, wg, wu = z(5, 64), z(24, 64), z(24, 64)
    assert fg.gated_f16(x, wg, wu).shape == (5, 24)
    h, g, u = fg.gated_f16(x, wg, wu, "gelu_tanh", save=True)
    assert h.shape == g.shape == u.shape == (5, 24)
    dx, dwg, dwu = fg.gated_f16_backward(h, x, wg, wu, g, u)
    assert dx.shape == (5, 64) and dwg.shape == dwu.shape == (24, 64)
    assert fg.recorder.calls == ["gated_f16", "gated_f16", "gated_f16_backward"]
    bad = [
        (lambda: fg.gated_f16(x.float(), wg, wu), ValueError, "fp16 or bf16"),
        (lambda: fg.gated_f16(x, wg.half(), wu), ValueError, "wg"),
        (lambda: fg.gated_f16(x, wg, z(32, 64)), ValueError, "wu"),
        (lambda: fg.gated_f16(x, z(24, 32), wu), ValueError, "wg"),
        (lambda: fg.gated_f16(x, wg, wu, out=z(5, 23)), ValueError, "out"),
        (lambda: fg.gated_f16(x, wg, wu, g=z(5, 24)), ValueError, "both or neither"),
        (lambda: fg.gated_f16(x, wg, wu, g=z(5, 24), u=z(5, 24).half()), ValueError, "u"),
        (lambda: fg.gated_f16(x, wg, wu, "relu"), KeyError, "relu"),
        (lambda: fg.gated_f16_backward(z(4, 24), x, wg, wu, g, u), ValueError, "dh"),
        (lambda: fg.gated_f16_backward(h, x, wg, wu, g, u.half()), ValueError, "u"),
        (lambda: fg.gated_f16_backward(h, x, wg, wu, g, u, dx=z(5, 24)), ValueError, "dx"),
        (lambda: fg.gated_f16_backward(h, x, wg, wu, g, u, workspace=z(8)), ValueError, "workspace"),
    ]
    for call, exc, match in bad:
        with pytest.raises(exc, match=match):
            call()
    assert len(fg.recorder.calls) == 3


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_binding_gemv(fg, fmt):
    N, K = 30, 192
    x, wq = z(3, K), z(N, K // 2, dtype=torch.uint8)
    shape, dt = fg.fp4_sf_shape(N, K, fmt)
    sf = torch.zeros(shape, dtype=dt)
    assert fg.gemv_fp4(x, wq, sf, fmt).shape == (3, N)
    assert fg.gated_gemv_fp4(x.half(), wq, sf, wq, sf, fmt).dtype == torch.float16
    bad = [
        (lambda: fg.gemv_fp4(x.float(), wq, sf, fmt), "fp16 or bf16"),
        (lambda: fg.gemv_fp4(x, wq[:, :64], sf, fmt), "wq"),
        (lambda: fg.gemv_fp4(x, wq, sf[:1, :4], fmt), "sf"),
        (lambda: fg.gemv_fp4(x, wq, sf, fmt, out=z(3, N, dtype=torch.float32)), "out"),
        (lambda: fg.gated_gemv_fp4(x, wq, sf, wq[:-1], sf, fmt), "wuq"),
        (lambda: fg.gated_gemv_fp4(x, wq, sf, wq, sf[:, :-4], fmt), "sfu"),
    ]
    for call, match in bad:
        with pytest.raises(ValueError, match=match):
            call()
    assert fg.recorder.calls == ["gemv_fp4", "gated_gemv_fp4"]


def test_non_contiguous_tensors_are_refused():
    from fine_grained_fp8_persistent_gb300 import binding

    class Fake:
        is_cuda = True

        def is_contiguous(self):
            return False

        def get_device(self):
            return 0
    with pytest.raises(ValueError, match="contiguous"):
        binding._launch("gemv_fp4", None, (Fake(),), ())
    with pytest.raises(ValueError, match="CUDA device"):
        binding._launch("gemv_fp4", None, (z(2, 2),), ())


def test_package_exports():
    import fine_grained_fp8_persistent_gb300 as pkg
    for name in ("gated_f16", "gated_f16_backward", "gated_backward_ws_bytes", "gemv_fp4", "gated_gemv_fp4"):
        assert callable(getattr(pkg, name))
    assert pkg.GEMV_MAX_ROWS == 16

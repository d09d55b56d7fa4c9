"""CPU checks of sizes near the end of 32 bits: the gated and matrix-vector operators round
sizes up to tiles in 32-bit integers, so what would pass their end is refused."""
import ctypes

import pytest

P, I = ctypes.c_void_p, ctypes.c_int
AL = P(0x10000)                       # never dereferenced: every call below is refused first
MOST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def lib():
    from fine_grained_fp8_persistent_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.fgf8_last_error.restype = ctypes.c_char_p
    lib.gated_f16.argtypes = [P] * 6 + [I] * 5 + [P]
    lib.gated_f16_backward.argtypes = [P] * 10 + [I] * 5 + [P]
    lib.gemv_fp4.argtypes = [P] * 4 + [I] * 5 + [P]
    lib.gated_gemv_fp4.argtypes = [P] * 6 + [I] * 6 + [P]
    return lib


def _calls(lib):
    yield lambda M, N, K: lib.gated_f16(AL, AL, AL, AL, None, None, M, N, K, 0, 0, None), True, 8
    yield lambda M, N, K: lib.gated_f16_backward(*[AL] * 10, M, N, K, 0, 0, None), True, 8
    yield lambda M, N, K: lib.gemv_fp4(*[AL] * 4, M, N, K, 0, 0, None), False, 64
    yield lambda M, N, K: lib.gated_gemv_fp4(*[AL] * 6, M, N, K, 0, 0, 0, None), False, 64


def test_sizes_past_the_last_tile_are_refused(lib):
    for call, many_rows, step in _calls(lib):
        over = MOST + step
        cases = [(1, over, 64), (1, 64, over)] + ([(over, 64, 64), (2 ** 31 - 1, 64, 64)] if many_rows else [])
        for M, N, K in cases:
            assert call(M, N, K) == 2, (M, N, K)
            assert str(MOST) in lib.fgf8_last_error().decode()


def test_the_largest_sizes_pass_that_check(lib):
    for call, many_rows, _ in _calls(lib):
        for M, N, K in [(1, MOST, 64), (1, 64, MOST)] + ([(MOST, 64, 64)] if many_rows else []):
            call(M, N, K)
            assert "sizes above" not in lib.fgf8_last_error().decode(), (M, N, K)

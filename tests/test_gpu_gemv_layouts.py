"""GPU tests of the matrix-vector kernels on every kind of layout that large weights run on:
several rounds of tiles per CTA, X in several pieces, the reduction split over clusters of
2, 4 and 8, and these together.  last_tile() tells which layout ran, so that other planning
constants cannot move a case off the layout it is here for unnoticed."""
import pytest
import torch

import fp4_weights as fp4
import gated_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _sums(x, w):
    x = x.double()
    return x @ w.t(), ref.gamma(x.shape[1]) * (x.abs() @ w.abs().t())


def test_last_tile_names_the_matrix_vector_launch(fg, dev):
    x = torch.ones(1, 64, dtype=torch.bfloat16, device=dev)
    for fmt, kind in ((0, "mxf4"), (1, "nvf4")):
        wq, sf, _ = fp4.random_matrix(48, 64, fmt, 1, dev)
        fg.gemv_fp4(x, wq, sf, fmt)
        assert fg.last_tile() == f"{kind} gemv 1x8 shallow r1 p1"
        fg.gated_gemv_fp4(x.expand(9, 64).contiguous(), wq, sf, wq, sf, fmt)
        assert fg.last_tile() == f"{kind} gated_gemv 1x16 deep r1 p1"
    w = torch.ones(48, 64, dtype=torch.bfloat16, device=dev)
    fg.gemm_f16(torch.ones(128, 64, dtype=torch.bfloat16, device=dev), torch.ones(128, 64, dtype=torch.bfloat16, device=dev))
    assert fg.last_tile().startswith("f16 dense")
    fg.gated_f16(x, w, w)
    assert fg.last_tile().startswith("f16 gated_gemv 1x8")


# (format, gated, bf16, M, N, K) and the layout that it is here for.  Odd N throughout; r: rounds
# of tiles, p: pieces of X.
LAYOUTS = [
    # X in pieces, one round
    (1, False, False, 16, 9619, 3328, "1x16 deep r1 p2"),
    (1, True, False, 5, 2321, 8448, "1x8 deep r1 p2"),
    (1, False, True, 16, 32771, 7168, "1x16 deep r1 p2"),
    (1, False, True, 7, 9647, 6272, "2x8 deep r1 p2"),
    (1, True, False, 15, 2341, 9664, "2x16 deep r1 p2"),
    (1, False, True, 8, 4173, 9600, "4x8 deep r1 p2"),
    (1, True, False, 8, 2121, 9344, "4x8 deep r1 p2"),
    # rounds, X staged once
    (0, False, False, 16, 40681, 64, "1x16 deep r2 p1"),
    (0, False, True, 8, 45001, 1280, "1x8 deep r2 p1"),
    (0, True, True, 8, 19739, 320, "1x8 deep r2 p1"),
    (1, True, False, 9, 19557, 1280, "1x16 deep r2 p1"),
    # rounds that each stage X again
    (0, False, False, 16, 44049, 4672, "1x16 deep r2 p2"),
    (1, True, True, 8, 35593, 2368, "1x8 deep r2 p2"),
    # a cluster that shares the reduction, in rounds
    (0, False, True, 16, 20313, 5184, "2x16 deep r2 p1"),
    (0, True, True, 16, 10471, 4608, "2x16 deep r2 p1"),
    (0, False, True, 16, 10203, 5696, "4x16 deep r2 p1"),
    (0, True, True, 16, 4877, 5696, "4x16 deep r2 p1"),
    # the same with X in pieces
    (1, False, True, 8, 44101, 11264, "2x8 deep r3 p2"),
    (1, True, False, 16, 20771, 9536, "2x16 deep r3 p2"),
    # clusters of one round
    (0, False, False, 13, 17, 5440, "8x16 deep r1 p1"),
    (1, False, True, 8, 297, 1856, "8x8 shallow r1 p1"),
    (1, True, True, 1, 15, 3712, "8x8 deep r1 p1"),
    (1, False, True, 6, 639, 896, "4x8 shallow r1 p1"),
    (0, False, True, 8, 1497, 448, "2x8 shallow r1 p1"),
    (0, True, False, 16, 1201, 16448, "8x16 deep r1 p1"),
]


@pytest.mark.parametrize("fmt,gated,bf16,M,N,K,layout", LAYOUTS)
def test_every_kind_of_layout(fg, dev, fmt, gated, bf16, M, N, K, layout):
    dtype = torch.bfloat16 if bf16 else torch.float16
    gen = torch.Generator(device=dev).manual_seed(N)
    x = torch.randn(M, K, generator=gen, device=dev)
    x[:, :: K // 5] *= 30.0
    x = x.to(dtype)
    wq, sf, w = fp4.random_matrix(N, K, fmt, N + K, dev)
    y, dy = _sums(x, w)
    del w
    R, T = ref.unit(dtype)
    kind = "nvf4" if fmt else "mxf4"
    if not gated:
        got = fg.gemv_fp4(x, wq, sf, fmt)
        assert fg.last_tile() == f"{kind} gemv {layout}"
        ref.close(got, y, dy + R * (y.abs() + dy) + T)
        assert torch.equal(got, fg.gemv_fp4(x, wq, sf, fmt))
        return
    uq, us, w = fp4.random_matrix(N, K, fmt, N + K + 1, dev)
    u, du = _sums(x, w)
    del w
    got = fg.gated_gemv_fp4(x, wq, sf, uq, us, fmt)
    assert fg.last_tile() == f"{kind} gated_gemv {layout}"
    ref.close(got, *ref.gate64(y, dy, u, du, "silu", dtype))
    assert torch.equal(got, fg.gated_gemv_fp4(x, wq, sf, uq, us, fmt))


@pytest.mark.parametrize("fmt", [0, 1])
def test_rows_kept_in_bf16_in_every_piece_and_round(fg, dev, fmt):
    """Small x beside large ones in one row and one chunk of each piece of X, in a layout that
    stages pieces again in every round of a cluster: the chunks in bf16 are those and no others."""
    M, N, K = (8, 44101, 11264) if fmt else (16, 28673, 8192)
    x = torch.randn(M, K, generator=torch.Generator(device=dev).manual_seed(3), device=dev)
    wq, sf, w = fp4.random_matrix(N, K, fmt, 4, dev)
    for k in range(0, K, 1024):
        x[(k // 1024) % M, k] = 2.0 ** 50
    x = x.to(torch.bfloat16)
    # weight zero under the large x, so that the others are the whole sum
    wq[:, 0:K // 2:512] &= 0xF0
    w[:, ::1024] = 0.0
    y, dy = _sums(x, w)
    R, T = ref.unit(x.dtype)
    got = fg.gemv_fp4(x, wq, sf, fmt)
    rounds, pieces = fg.last_tile().split()[-2:]
    if fmt:
        assert (rounds, pieces) == ("r3", "p2")
    ref.close(got, y, dy + R * (y.abs() + dy) + T)


# the 16-bit form of up to 16 tokens: (M, N, K) and layout
LAYOUTS16 = [
    (1, 2048, 7168, "1x8 deep r1 p1"),
    (5, 1032, 7176, "4x8 deep r1 p1"),
    (8, 2048, 7168, "4x8 deep r1 p1"),
    (16, 2048, 7168, "4x16 deep r1 p1"),
    (16, 600, 16392, "8x16 deep r1 p1"),
    (9, 9000, 8200, "2x16 deep r1 p1"),
    (16, 9000, 8200, "2x16 deep r1 p2"),
    (3, 40008, 136, "1x8 deep r3 p1"),
    (16, 40008, 1032, "1x16 deep r3 p1"),
    (16, 30000, 4104, "1x16 deep r2 p2"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,layout", LAYOUTS16)
def test_every_kind_of_layout_in_16_bits(fg, dev, M, N, K, layout, dtype):
    gen = torch.Generator(device=dev).manual_seed(N)
    x = torch.randn(M, K, generator=gen, device=dev).to(dtype)
    wg, wu = (torch.randn(N, K, generator=gen, device=dev).div_(K ** 0.5).to(dtype) for _ in range(2))
    want, bound = ref.forward64(x, wg, wu, "gelu_tanh")
    got = fg.gated_f16(x, wg, wu, "gelu_tanh", save=True)
    assert fg.last_tile() == f"f16 gated_gemv {layout}"
    for t, w, b, what in zip(got, want, bound, "hgu"):
        ref.close(t, w, b, what)
    again = fg.gated_f16(x, wg, wu, "gelu_tanh", save=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))

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

"""GPU tests of the gated block on the layouts that large sizes run on: pipelines that wrap
around, several tiles per cluster, accumulators used again, and the choice among the forms."""
import pytest
import torch

import gated_reference as ref
from test_gpu_gated import TYPES, _grad_inputs, _inputs, dev, fg  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_tile_of_another_kernel_changes_nothing(fg, dev, monkeypatch):
    """FGF8_FORCE_TILE names a tile of one kernel; the gated block keeps its own choice unless
    the tile is one of its own."""
    x, wg, wu = _inputs(64, 512, 1024, torch.bfloat16, 1, dev)
    want = fg.gated_f16(x, wg, wu)
    own = fg.last_tile()
    assert own.startswith("f16 gated_thin")
    for tile in ("2x224", "1x128ws", "", "9x9", "nonsense"):
        monkeypatch.setenv("FGF8_FORCE_TILE", tile)
        got = fg.gated_f16(x, wg, wu)
        assert fg.last_tile() == own and torch.equal(got, want), tile
    for tile in ("2x256", "1x128", "1x64"):
        monkeypatch.setenv("FGF8_FORCE_TILE", tile)
        fg.gated_f16(x, wg, wu)
        assert fg.last_tile() == f"f16 gated {tile}"


# reductions of many times the ring, for every number of CTAs that share it
THIN = [(17, 2048, 7168, "4x32"), (33, 2048, 7176, "4x48"), (64, 2048, 7168, "4x64"), (100, 5520, 7256, "3x112"),
        (200, 1032, 7168, "6x208"), (256, 2048, 7168, "4x256"), (256, 264, 16392, "8x256"), (40, 9000, 4104, "1x48")]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,tile", THIN)
def test_thin_rings_wrap_around(fg, dev, M, N, K, tile, dtype):
    x, wg, wu = _inputs(M, N, K, dtype, M, dev)
    want, bound = ref.forward64(x, wg, wu, "silu")
    got = fg.gated_f16(x, wg, wu, save=True)
    assert fg.last_tile() == f"f16 gated_thin {tile}"
    for t, w, b, what in zip(got, want, bound, "hgu"):
        ref.close(t, w, b, what)
    for _ in range(4):
        assert torch.equal(got[0], fg.gated_f16(x, wg, wu))
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("M", [17, 31, 47])
def test_thin_tokens_that_leave_a_warp_apart(fg, dev, M):
    """Odd token counts on one CTA per tile: the half-warps of the last pass have unlike work
    before the cluster meets."""
    for N, K in [(72, 64), (9728, 64)]:
        x, wg, wu = _inputs(M, N, K, torch.float16, 2, dev)
        want, bound = ref.forward64(x, wg, wu, "silu")
        got = fg.gated_f16(x, wg, wu)
        assert fg.last_tile().startswith("f16 gated_thin 1x")
        ref.close(got, want[0], bound[0])
    assert fg.check_status()[0] == 0


# M, N, K with several tiles per cluster on each tile: whole waves and a remainder, forward
# and backward (dX first, then dWg and dWu, with and without early ones)
MANY = [(2100, 4104, 1032), (4104, 2056, 2056), (5000, 3000, 1032), (4104, 1032, 8200)]


@pytest.mark.parametrize("tile", ["2x256", "1x128", "1x64"])
@pytest.mark.parametrize("M,N,K", MANY)
def test_many_tiles_per_cluster(fg, dev, monkeypatch, M, N, K, tile):
    dtype = torch.bfloat16 if tile != "1x128" else torch.float16
    dh, x, wg, wu, g, u = _grad_inputs(M, N, K, dtype, 13, dev)
    monkeypatch.setenv("FGF8_FORCE_TILE", tile)
    got = fg.gated_f16(x, wg, wu, "gelu_tanh", save=True)
    assert fg.last_tile() == f"f16 gated {tile}"
    for t, w, b, what in zip(got, *ref.forward64(x, wg, wu, "gelu_tanh"), "hgu"):
        ref.close(t, w, b, what)
    got = fg.gated_f16_backward(dh, x, wg, wu, g, u, "gelu_tanh")
    assert fg.last_tile() == f"f16 gated_grad {tile}"
    for t, w, b, what in zip(got, *ref.backward64(dh, x, wg, wu, g, u, "gelu_tanh"), ("dx", "dwg", "dwu")):
        ref.close(t, w, b, what)
    for _ in range(4):
        again = fg.gated_f16_backward(dh, x, wg, wu, g, u, "gelu_tanh")
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert fg.check_status()[0] == 0


def test_many_tiles_are_many():
    """The sizes above are what they are there for: on 152 SMs every tile gives clusters more than
    two tiles, and some a last tile of dX while the others start on the weights' gradients."""
    def up(a, b):
        return -(-a // b)
    uneven = 0
    for M, N, K in MANY:
        for ncta, bn in ((2, 256), (1, 128), (1, 64)):
            clusters = 152 // ncta
            assert up(M, 128 * ncta) * up(N, bn // 2) > 2 * clusters
            dx, dw = up(M, 128 * ncta) * up(K, bn), 2 * up(N, 128 * ncta) * up(K, bn)
            assert dx + dw > 2 * clusters
            uneven += dx > clusters and dx % clusters != 0
    assert uneven >= 8

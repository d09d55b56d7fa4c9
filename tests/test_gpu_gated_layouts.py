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

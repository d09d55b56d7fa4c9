"""GPU test that smoke() leaves the environment as it was."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [None, "1x16"])
def test_forced_tile_is_the_users_own(monkeypatch, value):
    import __graft_entry__
    monkeypatch.delenv("FGF8_FORCE_TILE", raising=False)
    if value is not None:
        monkeypatch.setenv("FGF8_FORCE_TILE", value)
    __graft_entry__.smoke()
    assert os.environ.get("FGF8_FORCE_TILE") == value

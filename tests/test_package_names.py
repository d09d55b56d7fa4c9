"""CPU test of the package's lazily found names."""
import pytest


def test_names_follow_binding(monkeypatch):
    import fine_grained_fp8_persistent_gb300 as pkg
    from fine_grained_fp8_persistent_gb300 import binding
    for name in ("gemv_fp4", "gemm_f16", "check_status"):
        assert getattr(pkg, name) is getattr(binding, name)
        other = object()
        monkeypatch.setattr(binding, name, other)
        assert getattr(pkg, name) is other
    monkeypatch.undo()
    assert pkg.gemv_fp4 is binding.gemv_fp4
    with pytest.raises(AttributeError):
        pkg.no_such_name

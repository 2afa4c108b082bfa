"""The library's C calls do not need the native binding: a machine without g++ or
Python's headers still loads and uses them (no GPU needed)."""
import pytest

from moe_grouped_gemm_nvfp4_gb300 import build
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F


def test_library_loads_where_the_binding_cannot_be_built(monkeypatch):
    def fail(verbose):
        raise RuntimeError("g++ failed on binding.cpp")

    monkeypatch.setattr(build, "_build_binding", fail)
    monkeypatch.setattr(build, "_binding_stale", lambda: True)
    monkeypatch.setattr(F, "_lib", None)
    monkeypatch.setattr(F, "_native", None)
    assert F.nvfp4_version() > 0
    assert F.nvfp4_status_string(0)
    with pytest.raises(RuntimeError, match="binding"):
        F.native()


def test_build_compiles_both(monkeypatch):
    made = []
    monkeypatch.setattr(build, "_build_binding", lambda verbose: made.append("binding"))
    monkeypatch.setattr(build, "_build_library", lambda verbose: made.append("library"))
    assert build.build(force=True) == build.LIB_PATH
    assert sorted(made) == ["binding", "library"]

"""What the build makes, for whom, and when it makes it again (no compiler is run here)."""
from pathlib import Path

import pytest
import torch

from paged_kv_cache_11_gb300 import _build, binding


def test_the_marshalling_is_made_for_one_python_and_torch(monkeypatch, tmp_path):
    made = []

    def run(cmd):
        made.append(cmd[cmd.index("-o") + 1])
        Path(made[-1]).touch()

    monkeypatch.setattr(_build, "LIBDIR", tmp_path)
    monkeypatch.setattr(_build, "_run", run)
    monkeypatch.setattr(_build, "_nvcc", lambda: "/opt/cuda/bin/nvcc")
    first = _build.build_marshal()
    assert _build.build_marshal() == first and len(made) == 1       # as it is
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    second = _build.build_marshal()
    assert second != first and len(made) == 2
    monkeypatch.setattr(binding.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert _build.build_marshal() not in (first, second) and len(made) == 3


def test_a_marshalling_of_other_versions_is_not_loaded(monkeypatch, tmp_path):
    monkeypatch.setattr(binding, "LIB_PATH", tmp_path / "libpagedkv.so")
    monkeypatch.setattr(binding, "_MARSHAL", None)
    (tmp_path / "_marshal.so").touch()
    (tmp_path / binding.marshal_name().replace(torch.__version__, "0.0.1")).touch()
    with pytest.raises(RuntimeError, match="not built"):
        binding._marshal()

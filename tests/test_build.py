"""What the build makes, for whom, and when it makes it again (no compiler is run here)."""
from pathlib import Path

import pytest
import torch

from paged_kv_cache_11_gb300 import _build, binding


def _refuse(*a, **k):
    raise AssertionError("not needed for the C library")


def test_the_c_library_needs_no_headers_of_torch(monkeypatch, tmp_path):
    ran = []

    def run(cmd):
        ran.append(cmd)
        Path(cmd[cmd.index("-o") + 1]).touch()

    monkeypatch.setattr(_build, "LIBDIR", tmp_path / "lib")
    monkeypatch.setattr(_build, "_run", run)
    monkeypatch.setattr(_build, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(_build, "build_marshal", _refuse)
    assert _build.build_library() == tmp_path / "lib" / "libpagedkv.so"
    assert len(ran) == len(_build.CUDA_SOURCES) + 1 and all(c[0] == "nvcc" for c in ran)
    home = str(Path(torch.__file__).resolve().parent)
    assert not any(home in word for c in ran for word in c)


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

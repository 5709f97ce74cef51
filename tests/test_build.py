"""The library's build does not depend on that of the tensor calls: without
PyTorch, or with a host compiler that fails on them, libdgemm.so is built all the
same, and the tensor calls say what is missing."""
import importlib.util
import os

import pytest

from dense_gemm_f32_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Build into a directory of its own, from one translation unit (quick)."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libdgemm.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_torch_binding.so"))
    monkeypatch.setattr(build, "UNITS", [("api.cu", "api", [])])
    return tmp_path


def _without_pytorch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def _without_a_compiler(monkeypatch):
    monkeypatch.setenv("CXX", os.path.join(os.sep, "nonexistent", "c++"))


def _failing_compiler(monkeypatch):
    monkeypatch.setenv("CXX", "false")


@pytest.mark.parametrize("broken", [_without_pytorch, _without_a_compiler, _failing_compiler])
def test_the_library_is_built_without_the_tensor_calls(broken, elsewhere, monkeypatch, capfd):
    broken(monkeypatch)
    lib = build.build()
    assert lib == build.LIB and os.path.exists(lib)
    assert not os.path.exists(build.BINDING)
    assert "tensor calls" in capfd.readouterr().err
    built = os.path.getmtime(lib)
    assert build.build() == lib and os.path.getmtime(lib) == built  # not built again for them
    with pytest.raises(RuntimeError, match="tensor calls"):
        build.build_binding()


def test_the_library_alone(elsewhere):
    assert os.path.exists(build.build_library())
    assert not os.path.exists(build.BINDING)

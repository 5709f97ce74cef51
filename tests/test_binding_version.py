"""The tensor calls are tied to the PyTorch and Python that they were compiled
against: another one has them rebuilt, and is refused until then."""
import os

import pytest

from dense_gemm_f32_gb300 import LibraryMissing, build, ops


@pytest.fixture
def built():
    build.build_binding()
    return build.BINDING


def test_another_version_is_stale(built, monkeypatch):
    assert not build.binding_stale()
    monkeypatch.setattr(build, "binding_key", lambda: "PyTorch 9.9.9, Python cpython-399, alpha")
    assert build.binding_stale()


def test_another_version_is_not_loaded(built, monkeypatch):
    monkeypatch.setattr(ops, "_binding", None)
    monkeypatch.setattr(build, "binding_key", lambda: "PyTorch 9.9.9, Python cpython-399, alpha")
    with pytest.raises(LibraryMissing, match="PyTorch 9.9.9"):
        ops._load()


def test_a_binding_without_a_record_is_stale(built, monkeypatch, tmp_path):
    copy = tmp_path / "_torch_binding.so"
    copy.write_bytes(b"")
    monkeypatch.setattr(build, "BINDING", str(copy))
    assert build.binding_stale()


def test_the_record_names_the_running_versions(built):
    import sys

    import torch

    key = build.binding_key()
    assert torch.__version__ in key and sys.implementation.cache_tag in key
    assert open(built + ".key", encoding="utf-8").read() == key
    assert os.path.exists(built)

"""What a build compiles again, and what it leaves in place when a part of it fails (CPU)."""
import os

import pytest

from paged_kv_cache_19_gb300 import build as cuda_build


@pytest.fixture
def small(monkeypatch, tmp_path):
    """A library of one host source and the binding, in a folder of their own."""
    monkeypatch.setattr(cuda_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(cuda_build, "LIB", str(tmp_path / "libkvpaged.so"))
    monkeypatch.setattr(cuda_build, "BINDING", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(cuda_build, "sources", lambda: [os.path.join(cuda_build.CSRC, "block_manager.cpp")])
    return tmp_path


def test_the_library_is_there_where_only_the_binding_fails(small, monkeypatch):
    """The calls that need no binding work without Python's and torch's headers."""
    monkeypatch.setattr(cuda_build, "BINDING_SRC", str(small / "missing.cpp"))
    with pytest.raises(RuntimeError, match="calls.cpp"):
        cuda_build.build()
    assert os.path.exists(cuda_build.LIB) and not os.path.exists(cuda_build.BINDING)
    before = os.path.getmtime(cuda_build.LIB)
    with pytest.raises((RuntimeError, OSError)):
        cuda_build.build()
    assert os.path.getmtime(cuda_build.LIB) == before        # and is not compiled again
    assert not cuda_build.up_to_date()


def test_another_torch_or_python_means_another_binding(small, monkeypatch):
    """File times say nothing about the headers a binary was compiled with."""
    import torch
    cuda_build.build()
    assert cuda_build.up_to_date()
    lib, binding = (os.path.getmtime(p) for p in (cuda_build.LIB, cuda_build.BINDING))
    cuda_build.build()
    assert (lib, binding) == tuple(os.path.getmtime(p) for p in (cuda_build.LIB, cuda_build.BINDING))
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert not cuda_build.up_to_date()
    cuda_build.build()
    assert cuda_build.up_to_date() and os.path.getmtime(cuda_build.BINDING) > binding
    assert os.path.getmtime(cuda_build.LIB) == lib

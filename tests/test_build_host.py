"""The build without PyTorch: the C library comes out, the tensor binding is left out and says so."""
import sys

import pytest

from packed_mm_rope_b200 import build


@pytest.fixture
def no_binding_yet(monkeypatch, tmp_path):
    """A built library, and a binding that would have to be built."""
    build.build_library()
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_tensors.so"))
    return tmp_path


def _without_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)       # import torch raises ImportError


def _torch_without_cuda(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.version, "cuda", None)


@pytest.mark.parametrize("missing", [_without_torch, _torch_without_cuda])
def test_library_is_built_alone(monkeypatch, capsys, no_binding_yet, missing):
    missing(monkeypatch)
    assert build.build_library() == build.LIB
    assert "_tensors.so left out: no PyTorch" in capsys.readouterr().err
    assert list(no_binding_yet.iterdir()) == []
    with pytest.raises(RuntimeError, match="without"):    # asked for by itself it is not left out silently
        build.build_binding()


def test_missing_compiler_and_broken_source(monkeypatch, capsys, no_binding_yet):
    pytest.importorskip("torch")
    monkeypatch.setattr(build, "_cxx", lambda: None)
    assert build.build_library() == build.LIB
    assert "no C++ compiler" in capsys.readouterr().err
    monkeypatch.undo()
    # what can be built and does not compile is an error, as before
    source = no_binding_yet / "binding.cpp"
    source.write_text("#error broken\n")
    monkeypatch.setattr(build, "BINDING", str(no_binding_yet / "_tensors.so"))
    monkeypatch.setattr(build, "BINDING_SOURCE", str(source))
    if build.binding_lacks() is None:
        with pytest.raises(RuntimeError, match="failed"):
            build.build_library()

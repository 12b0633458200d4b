"""The Python entry of the serving calls needs a C++ compiler and torch's headers; the library and its other calls do not,
so where they are missing the build says so and goes on (CPU only)."""
import shutil
import sys

import pytest

from bit_weight_only_tq_amd import build


@pytest.fixture
def stale(tmp_path, monkeypatch):
    """A binding of an earlier build, in a folder of its own."""
    f = tmp_path / "_serving.so"
    f.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "BINDING", str(f))
    return f


def _no_compiler(monkeypatch, tmp_path):
    monkeypatch.setattr(shutil, "which", lambda *a, **k: None)


def _no_torch(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setitem(sys.modules, "torch.utils", None)


def _no_torch_headers(monkeypatch, tmp_path):
    from torch.utils import cpp_extension
    monkeypatch.setattr(cpp_extension, "include_paths", lambda *a, **k: [str(tmp_path)])


def _no_python_headers(monkeypatch, tmp_path):
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})


@pytest.mark.parametrize("missing", [_no_compiler, _no_torch, _no_torch_headers, _no_python_headers])
def test_missing_needs_are_told_not_raised(missing, stale, monkeypatch, tmp_path, capsys):
    missing(monkeypatch, tmp_path)
    build._build_binding()
    assert "_serving.so not built" in capsys.readouterr().err
    assert not stale.exists()  # it was made for another library


def test_a_binding_that_does_not_compile_is_raised(stale, monkeypatch, tmp_path):
    (tmp_path / "binding.cpp").write_text("#error not C++ that compiles\n")
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    with pytest.raises(RuntimeError, match="not C\\+\\+ that compiles"):
        build._build_binding()

"""CPU tests of what the package needs to be built and called: the library needs hipcc alone; the
extension between torch and it is built where torch and a host compiler are, and done without
where it is missing."""
import os
import sys

import pytest
import torch

import semi_structured_sparse_amd as nm
from semi_structured_sparse_amd import build, decode


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A package folder of its own with an extension of an earlier build in it, and a library that
    is there at once."""
    monkeypatch.setattr(build, "PKG_DIR", str(tmp_path))
    (tmp_path / build.EXT_NAME).write_bytes(b"earlier")
    library = str(tmp_path / build.LIB_NAME)
    monkeypatch.setattr(build, "build_library", lambda verbose=False: library)
    return tmp_path


@pytest.mark.parametrize("missing", ["compiler", "torch", "headers"])
def test_the_library_is_built_without_what_the_extension_needs(place, monkeypatch, missing):
    if missing == "compiler":
        monkeypatch.setenv("CXX", "no-such-compiler")
    elif missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(torch, "__file__", str(place / "torch" / "__init__.py"))
    with pytest.warns(RuntimeWarning, match="_nmtorch"):
        assert build.build() == str(place / build.LIB_NAME)
    assert not (place / build.EXT_NAME).exists()      # of other sources than the library


def test_an_extension_that_does_not_compile_is_an_error(place, monkeypatch):
    monkeypatch.setattr(build, "extension_command", lambda out: [sys.executable, "-c", "raise SystemExit(3)"])
    with pytest.raises(RuntimeError, match="failed"):
        build.build()


def test_nothing_stands_against_the_extension_here():
    assert build.extension_obstacle() is None


def test_calls_do_without_the_extension(monkeypatch):
    """The checks of decode.py then make every call: the same errors, and one warning."""
    monkeypatch.setattr(decode, "_quick", None)
    monkeypatch.setitem(sys.modules, "semi_structured_sparse_amd._nmtorch", None)
    monkeypatch.delattr(nm, "_nmtorch", raising=False)
    x = torch.zeros(2, 3, 64, dtype=torch.float16)
    with pytest.warns(RuntimeWarning, match="_nmtorch.so"):
        with pytest.raises(ValueError, match="GPU"):
            nm.nm_rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    for name in decode._QUICK:
        assert getattr(decode._quick, name)() is NotImplemented
    assert os.path.exists(nm.LIB_PATH)

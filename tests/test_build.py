"""What the build does about the extension module: a missing host compiler, another torch."""
import os
import sys

import pytest

from block_scaled_w8a8_b200 import build as b


@pytest.fixture
def built(tmp_path, monkeypatch):
    """The library is there; the extension is to be built at a place of its own."""
    b.build()
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(b, "EXT_STAMP", str(tmp_path / "_torch_calls.stamp"))


def test_without_a_host_compiler_the_library_is_still_built(built, monkeypatch):
    monkeypatch.setenv("CXX", "/nowhere/c++")
    with pytest.warns(RuntimeWarning, match="is not built"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.EXT)


def test_another_torch_builds_the_extension_anew(built, monkeypatch):
    made = []

    def link(obj):
        made.append(obj)
        open(b.EXT, "w").close()

    monkeypatch.setattr(b, "_compile_ext", lambda: "torch_calls.o")
    monkeypatch.setattr(b, "_link_ext", link)
    b.build()
    b.build()
    assert len(made) == 1                   # the second time it is there
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    b.build()
    b.build()
    assert len(made) == 2


def test_without_torch_the_library_is_still_built(built, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)         # importing it raises
    with pytest.warns(RuntimeWarning, match="is not built"):
        assert b.build() == b.LIB


def test_an_extension_that_cannot_be_built_anew_does_not_stay(built, monkeypatch):
    """It would call the new library with the old arguments."""
    for f in (b.EXT, b.EXT_STAMP):
        open(f, "w").close()
    monkeypatch.setenv("CXX", "/nowhere/c++")
    with pytest.warns(RuntimeWarning, match="is not built"):
        b.build()
    assert not os.path.exists(b.EXT) and not os.path.exists(b.EXT_STAMP)

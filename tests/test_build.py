"""What build() makes, and of what: the library alone where there is no torch."""
import importlib.util

import pytest

from block_sparse_long_rope_b200 import build as star_build


def test_library_without_torch(monkeypatch):
    """The C ABI needs no torch: its build must not ask for it."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(star_build, "build_native", lambda force=False: pytest.fail("torch was asked for"))
    assert star_build.build() == star_build.LIB


def test_a_failing_native_half_is_an_error(monkeypatch):
    def fails(force=False):
        raise RuntimeError("no compiler")
    monkeypatch.setattr(star_build, "build_native", fails)
    with pytest.raises(RuntimeError, match="no compiler"):
        star_build.build()

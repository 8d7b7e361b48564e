"""The library is built for users of the C interface too, who need not have torch's headers."""

import os

import pytest

from bit_quantization_head_b200 import build


def small_build(monkeypatch, tmp_path):
    """One host file instead of all sources, into a folder of its own."""
    monkeypatch.setattr(build, "SOURCES", ["host_plan.cpp"])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkvtc.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))


def test_the_library_is_linked_where_the_bindings_half_cannot_be_built(monkeypatch, tmp_path):
    small_build(monkeypatch, tmp_path)

    def fails():
        raise RuntimeError("no headers here")

    monkeypatch.setattr(build, "_build_marshal", fails)
    (tmp_path / "_marshal.so").write_bytes(b"of an earlier build")
    with pytest.raises(RuntimeError, match="libkvtc.so is built.*no headers here"):
        build.build()
    assert os.path.getsize(tmp_path / "libkvtc.so") > 0
    assert not (tmp_path / "_marshal.so").exists()   # nothing of another build stays beside the library


def test_a_missing_torch_is_named(monkeypatch, tmp_path):
    small_build(monkeypatch, tmp_path)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    with pytest.raises(RuntimeError, match="libkvtc.so is built.*torch"):
        build.build()
    assert os.path.getsize(tmp_path / "libkvtc.so") > 0

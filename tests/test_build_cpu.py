"""The build without what only the extension module needs: the C library is
linked all the same, and the missing part is an error.  A script stands in for
hipcc."""

import os

import pytest

from cross_rank_collective_amd import build as b


@pytest.fixture
def fake(tmp_path, monkeypatch):
    cc = tmp_path / "hipcc"
    cc.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
    cc.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(cc))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libptored.so"))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "_torch_calls.so"))
    return tmp_path


@pytest.mark.parametrize("error", [RuntimeError("g++ failed"), ImportError("no torch"),
                                   FileNotFoundError("g++")])
def test_the_library_does_not_wait_for_the_extension(fake, monkeypatch, error):
    def compile_ext():
        raise error

    monkeypatch.setattr(b, "_compile_ext", compile_ext)
    with pytest.raises(type(error)):
        b.build(4)
    assert os.path.exists(b.LIB) and not os.path.exists(b.EXT)


def test_without_the_library_nothing_is_linked(fake, monkeypatch):
    def compile_unit(unit):
        raise RuntimeError("hipcc failed")

    monkeypatch.setattr(b, "_compile", compile_unit)
    monkeypatch.setattr(b, "_compile_ext", lambda: "unused.o")
    with pytest.raises(RuntimeError, match="hipcc failed"):
        b.build(4)
    assert not os.path.exists(b.LIB)

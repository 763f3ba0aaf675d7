"""CPU: libvocoder.so and the compiled binding for torch tensors are built apart from one another.

The compilers are stand-ins that write their output file and a line into a log."""
from __future__ import annotations

import os
import stat

import pytest

from dac_vocoder_decode_gb300 import build as B


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build into a folder of its own; `.ran()` lists the outputs that were compiled since the last
    look."""
    log = tmp_path / "log"
    log.write_text("")
    tool = tmp_path / "compiler"
    tool.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && out=$2; shift; done\n'
                    f'echo "$out" >> "{log}"\n: > "$out"\n')
    tool.chmod(tool.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(B, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib" / "libvocoder.so"))
    monkeypatch.setattr(B, "nvcc", lambda: str(tool))
    monkeypatch.setattr(B, "torch_dir", lambda: str(tmp_path))
    (tmp_path / "version.py").write_text("__version__ = '9.1.0+cu130'\n")
    monkeypatch.setattr(B, "torch_command", lambda out: [str(tool), "-o", out])

    class Place:
        path = tmp_path

        @staticmethod
        def ran():
            lines = log.read_text().split("\n")[:-1]
            log.write_text("")
            return lines
    return Place


def test_both_are_built_once(place):
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.torch_lib())
    assert len(place.ran()) == len([f for f in B.sources() if f.endswith(".cu")]) + 2
    B.build()
    assert place.ran() == []
    B.build(force=True)
    assert len(place.ran()) > 2
    assert not [f for f in os.listdir(B.LIBDIR) if "tmp" in f]


@pytest.mark.parametrize("command", [["false"], ["/nonexistent/compiler", "-o", "x"]])
def test_library_stands_where_the_binding_is_not_built(place, monkeypatch, command):
    monkeypatch.setattr(B, "torch_command", lambda out: command)
    with pytest.warns(RuntimeWarning, match="not built"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.torch_lib())
    place.ran()
    B.build()  # neither the library nor the vain attempt again
    assert place.ran() == [] and B.up_to_date()


def test_a_binding_of_older_sources_is_taken_out(place, monkeypatch):
    B.build()
    monkeypatch.setattr(B, "torch_command", lambda out: ["false"])
    with pytest.warns(RuntimeWarning, match="not built"):
        B.build(force=True)
    assert not os.path.exists(B.torch_lib())


def test_library_stands_without_torch(place, monkeypatch):
    monkeypatch.setattr(B, "torch_dir", lambda: None)
    B.build()
    assert os.listdir(B.LIBDIR) == ["libvocoder.so"] and B.up_to_date()


def test_a_failing_library_still_raises(place, monkeypatch):
    monkeypatch.setattr(B, "nvcc", lambda: "false")
    with pytest.raises(RuntimeError, match="libvocoder"):
        B.build()
    assert not os.path.exists(B.LIB)


def test_the_binding_is_for_one_python_and_torch(place):
    B.build()
    first = B.torch_lib()
    place.ran()
    (place.path / "version.py").write_text("__all__ = ['__version__', 'cuda']\n__version__: str = '9.2.0'\n")
    assert B.torch_version() == "9.2.0"
    assert not os.path.exists(B.torch_lib()) and not B.up_to_date()
    B.build()
    assert place.ran() and os.path.exists(B.torch_lib()) and B.torch_lib() != first
    (place.path / "version.py").unlink()
    assert "unknown" in B.torch_lib()

"""The library and the compiled part of its Python binding are built apart: what the
binding lacks (a compiler, Python's or torch's headers) costs its five calls and nothing
else.  The compilers here are scripts that write empty files and their command lines."""
import importlib.metadata
import os
import stat

import pytest

from row_wise_softmax_warp_gb300 import binding, build

COMPILER = """#!/bin/sh
echo "$0 $@" >> "$BUILD_LOG"
[ -n "$BREAK" ] && case "$0 $*" in *$BREAK*) echo "no headers here" >&2; exit 1;; esac
while [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done
"""


@pytest.fixture
def tools(tmp_path, monkeypatch):
    for name in ("nvcc", "cxx"):
        path = tmp_path / name
        path.write_text(COMPILER)
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setenv(name.upper(), str(path))
    monkeypatch.setenv("BUILD_LOG", str(tmp_path / "log"))
    for name, at in (("BUILD", "build"), ("LIB", "librowops.so"), ("HOST", "_host.so")):
        monkeypatch.setattr(build, name, str(tmp_path / at))

    def commands():
        log = tmp_path / "log"
        lines = log.read_text().splitlines() if log.exists() else []
        log.write_text("")
        return sum("/nvcc " in x for x in lines), sum("/cxx " in x for x in lines)

    return commands


def test_built_once(tools, recwarn):
    assert build.build() == build.LIB and os.path.exists(build.LIB) and os.path.exists(build.HOST)
    assert tools() == (len(build._sources()) + 1, 1) and not recwarn
    build.build()
    assert tools() == (0, 0)
    build.build(force=True)
    assert tools() == (len(build._sources()) + 1, 1)


@pytest.mark.parametrize("lacking", ["compiler", "headers", "torch's record"])
def test_the_library_needs_no_binding(tools, monkeypatch, lacking):
    if lacking == "compiler":
        monkeypatch.setenv("CXX", "/nowhere/cxx")
    elif lacking == "headers":
        monkeypatch.setenv("BREAK", "/cxx ")
    else:
        def none(name):
            raise importlib.metadata.PackageNotFoundError(name)
        monkeypatch.setattr(importlib.metadata, "version", none)
    with open(build.HOST, "w") as f:
        f.write("of an older library")
    with pytest.warns(RuntimeWarning, match="binding"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)
    assert not os.path.exists(build.HOST)  # its calls may have changed
    assert tools()[0] == len(build._sources()) + 1
    with pytest.warns(RuntimeWarning, match="binding"):
        build.build()
    assert tools()[0] == 0  # the library is not compiled again


def test_a_broken_library_is_an_error(tools, monkeypatch):
    monkeypatch.setenv("BREAK", "dropout.cu")
    with pytest.raises(RuntimeError, match="dropout.cu"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_calls_without_the_binding_say_so(monkeypatch):
    """They raise, and calls of the library itself do not."""
    monkeypatch.setattr(binding, "_host", None)
    monkeypatch.setattr(binding, "library", lambda: None)
    monkeypatch.setitem(__import__("sys").modules, "row_wise_softmax_warp_gb300._host", None)  # as if it were not there
    import row_wise_softmax_warp_gb300 as pkg
    monkeypatch.delattr(pkg, "_host", raising=False)
    with pytest.raises(RuntimeError, match="compiled part of the binding"):
        binding._native()

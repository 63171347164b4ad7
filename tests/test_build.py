"""The build script's decisions, with the compilers replaced: what is stale, and
what is left where torch's headers are missing."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_segment_b200 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the script's paths; compilers that write their output's name, recorded."""
    csrc = tmp_path / "pkg" / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "a.cu").write_text("")
    (csrc / "serve_ext.cpp").write_text("")
    for name, at in (("HERE", "pkg"), ("CSRC", "pkg/csrc"), ("LIB", "pkg/libtfpaged.so"), ("EXT", "pkg/_serve.so"),
                     ("EXT_FOR", "pkg/_serve.built"), ("EXT_SRC", "pkg/csrc/serve_ext.cpp")):
        monkeypatch.setattr(b, name, str(tmp_path / at))
    ran = []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        ran.append(os.path.basename(out))
        open(out, "w").close()

    monkeypatch.setattr(subprocess, "run", run)
    return ran


def test_the_library_alone_needs_nothing_of_torch(tree, monkeypatch):
    monkeypatch.setattr(b, "compile_ext", lambda obj: pytest.fail("compiled the extension"))
    assert b.build(ext=False) == b.LIB and tree == ["a.cu.o", "libtfpaged.so"]
    assert not b.stale(ext=False) and b.stale()
    assert b.build(ext=False) == b.LIB and len(tree) == 2  # nothing to do


def test_an_extension_that_does_not_compile_leaves_the_library(tree, monkeypatch):
    def missing(obj):
        raise subprocess.CalledProcessError(1, "g++")

    monkeypatch.setattr(b, "compile_ext", missing)
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert os.path.exists(b.LIB) and not b.stale(ext=False) and b.stale()


def test_another_torch_or_python_makes_the_extension_stale(tree, monkeypatch):
    b.build()
    assert sorted(tree) == ["_serve.so", "a.cu.o", "libtfpaged.so", "serve_ext.o"] and not b.stale()
    monkeypatch.setattr(b, "ext_for", lambda: "python 3.11 torch 2.0")
    assert b.stale() and not b.stale(ext=False)
    b.build()
    assert not b.stale()
    os.utime(b.EXT_SRC, (os.path.getmtime(b.EXT) + 5,) * 2)
    assert b.stale() and not b.stale(ext=False)


def test_the_script_runs_without_the_package():
    """--lib-only is a file to run: importing it brings in neither torch nor the package."""
    code = ("import importlib.util, sys; s = importlib.util.spec_from_file_location('b', sys.argv[1]); "
            "m = importlib.util.module_from_spec(s); s.loader.exec_module(m); assert 'torch' not in sys.modules")
    assert subprocess.call([sys.executable, "-c", code, b.__file__]) == 0

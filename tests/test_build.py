"""CPU checks of the build: the library for C callers does not depend on torch or on its headers."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_25_gb300 import build


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """A compiler that only makes its output file; .fail: a source it does not compile."""
    class Compiler:
        fail, made = "nothing", []

        def run(self, cmd, **kw):
            if any(self.fail in a for a in cmd):
                return subprocess.CompletedProcess(cmd, 1, "", "no such header")
            out = cmd[cmd.index("-o") + 1]
            self.made.append(os.path.basename(out).split(".so")[0])
            open(out, "w").close()
            return subprocess.CompletedProcess(cmd, 0, "", "")

    c = Compiler()
    c.made = []
    monkeypatch.setattr(build.subprocess, "run", c.run)
    monkeypatch.setattr(build, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "OUT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpa.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_pa_marshal.so"))
    return c


def test_without_torch_the_library_is_built(compiler, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)          # import torch raises ImportError
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
    compiler.made.clear()
    build.build()                                            # and is up to date then
    assert not compiler.made


def test_without_torchs_headers_the_library_is_built_first(compiler):
    compiler.fail = "marshal.cpp"
    with pytest.raises(RuntimeError, match="marshal"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
    compiler.fail = "nothing"
    compiler.made.clear()
    build.build()                                            # only what is missing
    assert os.path.exists(build.MARSHAL) and "libpa" not in compiler.made


def test_what_is_built_is_not_built_again(compiler):
    build.build()
    assert {"libpa", "_pa_marshal"} <= set(compiler.made)
    compiler.made.clear()
    build.build()
    assert not compiler.made
    build.build(force=True)
    assert {"libpa", "_pa_marshal"} <= set(compiler.made)


def test_a_source_that_does_not_compile_raises(compiler):
    compiler.fail = "decode.cu"
    with pytest.raises(RuntimeError, match="decode.cu"):
        build.build()
    assert not os.path.exists(build.LIB)

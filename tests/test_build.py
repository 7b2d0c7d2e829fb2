"""What build() needs: ROCm for libgdr.so, and more only for the Python extension.  A stand-in for
hipcc writes the library; the extension's source is one that compiles at once, or not at all."""
import os
import stat

import pytest

from gated_delta_rule_70_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho library > "$2"\n')
    hipcc.chmod(hipcc.stat().st_mode | stat.S_IXUSR)
    (tmp_path / "binding.cpp").write_text("#include <Python.h>\n")
    for name, value in (("hipcc", lambda: str(hipcc)), ("SOURCES", ["one.hip"]), ("CSRC", str(tmp_path)),
                        ("OBJ_DIR", str(tmp_path / "obj")), ("LIB", str(tmp_path / "libgdr.so")),
                        ("BINDING", str(tmp_path / "_binding.so"))):
        monkeypatch.setattr(build, name, value)
    (tmp_path / "_binding.so").write_text("of other sources")
    return tmp_path


def test_everything_there(tree):
    assert build.build(verbose=False) == str(tree / "libgdr.so") and os.path.exists(build.LIB)
    assert (tree / "_binding.so").read_bytes() != b"of other sources"


def test_no_compiler(tree, monkeypatch, capfd):
    empty = tree / "empty"
    empty.mkdir()
    monkeypatch.setattr(build, "hipcc", lambda: "/bin/sh")      # by its path, as hipcc is found
    monkeypatch.setattr(build, "_compile", lambda src: "")
    monkeypatch.setattr(build.subprocess, "run", link_only(build.subprocess.run))
    monkeypatch.setenv("PATH", str(empty))
    build.build(verbose=False)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "compiler" in capfd.readouterr().err


def link_only(run):
    def link(cmd, **kw):
        if build.LIB + ".tmp" not in cmd:
            return run(cmd, **kw)
        open(build.LIB + ".tmp", "w").close()
    return link


@pytest.mark.parametrize("header", ["Python.h", "torch/csrc/autograd/python_variable.h"])
def test_no_headers(tree, monkeypatch, capfd, header):
    from torch.utils import cpp_extension

    if header == "Python.h":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tree / "none")})
    paths = [p for p in cpp_extension.include_paths() if not os.path.exists(os.path.join(p, header))]
    monkeypatch.setattr(cpp_extension, "include_paths", lambda *a: paths)
    (tree / "binding.cpp").write_text(f"#include <{header}>\n")
    build.build(verbose=False)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert header in capfd.readouterr().err


def test_extension_that_does_not_compile(tree):
    """That is an error, but not the library's."""
    (tree / "binding.cpp").write_text("no C++\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build(verbose=False)
    assert os.path.exists(build.LIB)

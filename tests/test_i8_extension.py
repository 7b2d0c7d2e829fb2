"""The 8-bit operators where their Python extension is not built, or built from other sources."""
import shutil
import subprocess
import sysconfig

import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gated_delta_rule_70_amd import quantized as qz


def calls():
    x, q8 = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8)
    yield lambda: gdr.add_rmsnorm_i8(x, torch.zeros(64))
    yield lambda: gdr.gated_rmsnorm_i8(x.view(2, 1, 64), x.view(2, 1, 64), torch.zeros(64))
    yield lambda: gdr.matmul_i8(q8, torch.zeros(2), q8, torch.zeros(2))


def test_without_the_extension(tmp_path, monkeypatch):
    """Every call goes through Python (as far as CPU tensors get there), and the first one says so."""
    monkeypatch.setattr(qz, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(qz, "_B", None)
    first, *others = calls()
    with pytest.warns(RuntimeWarning, match="not built"), pytest.raises(ValueError, match="GPU tensor"):
        first()
    for call in others:
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_extension_of_other_sources(tmp_path, monkeypatch):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = tmp_path / "binding.c", tmp_path / "_binding.so"
    src.write_text("#include <Python.h>\nstatic PyModuleDef d = {PyModuleDef_HEAD_INIT, \"_binding\", 0, -1, 0};\n"
                   "PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&d); }\n")
    subprocess.run([cc, "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(qz, "BINDING_PATH", str(so))
    monkeypatch.setattr(qz, "_B", None)
    with pytest.raises(RuntimeError, match="rebuild it"):
        next(calls())()
    assert qz._B is None

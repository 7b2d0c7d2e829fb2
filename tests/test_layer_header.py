"""Every function that gdr_layer.h declares, whatever it returns, is exported by the library and bound as declared."""
import ctypes
import re
import subprocess

import gated_delta_rule_70_amd as gdr
from test_layer_api import HEADER, L  # noqa: F401

RETURNS = {"int": ctypes.c_int, "size_t": ctypes.c_size_t}


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return {name: (ret, args) for ret, name, args in re.findall(r"^(\w+)\s+(gdr_\w+)\s*\(([^)]*)\)\s*;", src, re.M)}


def test_declared_functions():
    assert set(declared()) == {"gdr_causal_conv", "gdr_qk_norm_rope", "gdr_selective_scan", "gdr_selective_scan_step",
                               "gdr_selective_scan_workspace_bytes"}
    assert set(re.findall(r"\b(gdr_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S))) == set(declared())


def test_exported(L):  # noqa: F811
    out = subprocess.run(["nm", "-D", "--defined-only", gdr.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(declared()) <= set(re.findall(r"\bT\s+(\w+)$", out, re.M))


def test_bound(L):  # noqa: F811
    """One argument more than bound would be passed as a C int, and so would a stream's handle or a size."""
    for name, (ret, args) in declared().items():
        fn = getattr(L, name)
        assert fn.restype is RETURNS[ret], name
        kinds = [ctypes.c_size_t if a.split()[0] == "size_t" else ctypes.c_void_p if "*" in a else ctypes.c_int for a in args.split(",")]
        assert fn.argtypes == kinds, name

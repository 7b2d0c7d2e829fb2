"""Build libgdr.so (HIP kernels for gfx950 + the C-ABI host entry points) in-tree.

Usage: ``python -m gated_delta_rule_70_amd.build`` (or ``build()`` from Python).  Each
translation unit is compiled by hipcc in parallel, then linked into
``gated_delta_rule_70_amd/libgdr.so``.  The library links against the HIP runtime by
SONAME (libamdhip64.so.7), so inside a process that already loaded PyTorch's bundled
runtime it binds to that same runtime and shares its streams and device pointers.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdr.so")
BINDING = os.path.join(PKG, "_binding.so")

SOURCES = ["gdr_api.cpp", "decode.hip", "chunk_prep.hip", "chunk_prep_split.hip", "chunk_carry.hip",
           "chunk_carry_wide.hip", "tree_verify.hip", "varlen_plan.hip", "i8_api.cpp", "i8_norm.hip",
           "i8_matmul.hip"]
ARCH = os.environ.get("GDR_OFFLOAD_ARCH", "gfx950")

# Packed fp32 VALU forms are kept out of the device code (plain fp32 FMAs only).
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-Wno-unused-function", "-Wno-unused-variable", "-Wno-unused-but-set-variable"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libgdr.so)")


def _compile(src: str) -> str:
    out = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *COMMON, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stderr}")
    # the host pass does not know the gfx950 feature flag; that warning is expected
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in res.stderr.splitlines() if ln.strip() and noise not in ln]
    if msgs:
        print("\n".join(msgs), file=sys.stderr)
    return out


def _cxx():
    return shutil.which("g++") or shutil.which("c++")


def _binding_includes() -> list[str]:
    from torch.utils import cpp_extension

    return [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths()]


def _binding_lacks() -> str | None:
    """What the extension needs and this machine does not have.  libgdr.so needs none of it."""
    if not _cxx():
        return "a C++ compiler"
    try:
        paths = _binding_includes()
    except ImportError:
        return "PyTorch"
    for header in ("Python.h", "torch/csrc/autograd/python_variable.h"):
        if not any(os.path.exists(os.path.join(p, header)) for p in paths):
            return header
    return None


def _compile_binding() -> None:
    """The Python extension of the 8-bit operators (csrc/binding.cpp), host code against PyTorch's
    headers."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    paths = _binding_includes()
    tmp = BINDING + ".tmp"
    cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f for p in paths for f in ("-isystem", p)],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{res.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = True) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    lacks = _binding_lacks()
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 1)) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    if lacks:
        if os.path.exists(BINDING):
            os.remove(BINDING)  # of other sources
        print(f"{BINDING} needs {lacks} and was not built: the 8-bit operators' calls from Python take 3 to 5 us longer",
              file=sys.stderr)
    else:
        binding.result()
    return LIB


if __name__ == "__main__":
    build()

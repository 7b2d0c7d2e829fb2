"""The host entry points of the operators before and beside the recurrence under AddressSanitizer and
UndefinedBehaviorSanitizer, with the kernel launchers stubbed out (no GPU involved)."""
import os

import pytest

from test_sanitizers import CLANG, CSRC, ENV, HIPCC, INCLUDE, SAN, SAN_FLAGS, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not available")
def test_layer_entry_points_under_sanitizers(tmp_path):
    host_san = [f for flag in SAN_FLAGS for f in ("-Xarch_host", flag)]
    objs = []
    for src in (os.path.join(CSRC, "layer_api.cpp"), os.path.join(SAN, "stub_layer_launchers.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, "-O1", "-g", "-std=c++17", "--offload-arch=gfx950", *host_san, "-I", INCLUDE, "-I", CSRC,
              "-x", "hip", "-c", src, "-o", obj])
        objs.append(obj)
    drv = str(tmp_path / "api_layer_driver.o")
    _run([CLANG, "-O1", "-g", "-std=c99", *SAN_FLAGS, "-I", INCLUDE, "-c", os.path.join(SAN, "api_layer_driver.c"), "-o", drv])
    exe = str(tmp_path / "api_layer_san")
    _run([HIPCC, "--offload-arch=gfx950", *host_san, drv, *objs, "-o", exe])
    res = _run([exe], env=ENV, timeout=300)
    assert "layer api sanitize ok" in res.stdout

"""A libgdr.so that was built from other sources is refused with what to do about it, whatever it
lacks: another version, or symbols that this package binds."""
import shutil
import subprocess

import pytest

import gated_delta_rule_70_amd as gdr

CC = shutil.which("gcc") or shutil.which("cc")


@pytest.mark.skipif(CC is None, reason="no C compiler")
@pytest.mark.parametrize("src", [
    f"int gdr_abi_version(void) {{ return {gdr.ABI_VERSION - 1}; }}",  # an older version, with fewer symbols
    f"int gdr_abi_version(void) {{ return {gdr.ABI_VERSION}; }} const char* gdr_status_str(int s) {{ return \"\"; }}",
    "int gdr_decode_step(void) { return 0; }",
], ids=["older", "symbols_missing", "no_version"])
def test_other_library(src, tmp_path, monkeypatch):
    c, so = tmp_path / "lib.c", tmp_path / "libgdr.so"
    c.write_text(src)
    subprocess.run([CC, "-shared", "-fPIC", "-o", str(so), str(c)], check=True)
    monkeypatch.setattr(gdr, "LIB_PATH", str(so))
    monkeypatch.setattr(gdr, "_lib", None)
    with pytest.raises(RuntimeError, match="rebuild it"):
        gdr.lib()
    assert gdr._lib is None

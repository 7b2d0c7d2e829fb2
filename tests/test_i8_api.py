"""Refusals of the 8-bit operators, on the host: the C entry points with fake device addresses
(only on calls whose validation fails, or that have no rows), and the Python binding with CPU
tensors, whose checks of shapes and types run before the device is looked at."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gated_delta_rule_70_amd import quantized as qz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdr_i8.h")
OK, ENULL, ESHAPE, EUNSUP, EALIGN, EALIAS = range(6)
BASE, SLOT = 1 << 40, 1 << 34


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gdr.LIB_PATH):
        from gated_delta_rule_70_amd import build

        build.build(verbose=False)
    return gdr.lib()


def addr(i, off=0):
    return BASE + i * SLOT + off


def test_library_exports_the_header(L):
    names = set(re.findall(r"^\s*int\s+(gdr_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == {"gdr_add_rmsnorm_i8", "gdr_gated_rmsnorm_i8", "gdr_matmul_i8"}
    out = subprocess.run(["nm", "-D", "--defined-only", gdr.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT\s+(\w+)$", out, re.M))


def test_limits_match_the_header():
    src = open(HEADER).read()
    for name, value in (("GDR_NORM_MAX_COLS", qz.NORM_MAX_COLS), ("GDR_MATMUL_I8_MAX_K", qz.MATMUL_I8_MAX_K),
                        ("GDR_MATMUL_I8_MAX_OUT", qz.MATMUL_I8_MAX_OUT)):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == value


def norm(L, entry="add", **kw):
    d = dict(rows=3, heads=1, cols=64, x_dtype=0, gate_dtype=0, weight_dtype=0, eps=1e-6, x_stride=64, r_stride=64,
             out_stride=64)
    p = dict(x=addr(0), r=addr(1), w=addr(2), q=addr(3), scale=addr(4), out=addr(5))
    if entry == "gated":
        d.update(heads=2, x_stride=128, r_stride=128)
    for k, v in kw.items():
        (d if k in d else p)[k] = v
    dims = qz.NormDims(**d)
    if entry == "gated":
        return L.gdr_gated_rmsnorm_i8(ctypes.addressof(dims), p["x"], p["r"], p["w"], p["q"], p["scale"], None)
    return L.gdr_add_rmsnorm_i8(ctypes.addressof(dims), p["x"], p["r"], p["w"], p["q"], p["scale"], p["out"], None)


@pytest.mark.parametrize("entry", ["add", "gated"])
def test_norm_refusals(L, entry):
    fn = L.gdr_add_rmsnorm_i8 if entry == "add" else L.gdr_gated_rmsnorm_i8
    assert fn(*[None] * (8 if entry == "add" else 7)) == ENULL
    for name in ("x", "w", "q", "scale") + (("r",) if entry == "gated" else ()):
        assert norm(L, entry, **{name: None}) == ENULL, name
    for kw in (dict(rows=-1), dict(rows=(1 << 30) + 1), dict(heads=0), dict(cols=0), dict(x_stride=-1), dict(r_stride=-1),
               dict(cols=32768 + 1) if entry == "add" else dict(heads=1025, cols=32),
               dict(rows=1 << 30, x_stride=1 << 40)):
        assert norm(L, entry, **kw) == ESHAPE, kw
    for kw in (dict(x_dtype=2), dict(weight_dtype=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(L, entry, **kw) == EUNSUP, kw
    for name, off in (("x", 1), ("r", 1), ("w", 1), ("scale", 2)) + ((("out", 1),) if entry == "add" else ()):
        assert norm(L, entry, **{name: addr(9, off)}) == EALIGN, name
    assert norm(L, entry, x_dtype=1, weight_dtype=1, x=addr(0, 2)) == EALIGN
    for kw in (dict(q=addr(0, 64)), dict(q=addr(1)), dict(q=addr(2, 8)), dict(scale=addr(0)), dict(scale=addr(2)),
               dict(scale=addr(3, 128)), dict(q=addr(0, -1))):
        assert norm(L, entry, **kw) == EALIAS, kw
    assert norm(L, entry, rows=0, x=None, r=None, w=None, q=None, scale=None) == OK


def test_add_rmsnorm_refusals(L):
    assert norm(L, heads=2) == ESHAPE
    assert norm(L, out_stride=63) == ESHAPE
    assert norm(L, x_dtype=1, weight_dtype=0) == EUNSUP
    # the new stream over x or the residual: only row for row
    for kw in (dict(out=addr(0), out_stride=72), dict(out=addr(0, 2)), dict(out=addr(1), r_stride=80), dict(out=addr(2)),
               dict(out=addr(3)), dict(out=addr(4)), dict(out=addr(0), r=addr(0, 64))):
        assert norm(L, **kw) == EALIAS, kw


def test_gated_rmsnorm_refusals(L):
    for c in (16, 48, 256):
        assert norm(L, "gated", cols=c) == EUNSUP
    assert norm(L, "gated", gate_dtype=7) == EUNSUP


def product(L, outs=(4, 5), out_cols=(32, 16), out_stride=None, bias=addr(3), null_outs=False, **kw):
    d = dict(M=5, K=64, n_out=len(outs), out_dtype=0, a_stride=64, w_stride=64)
    p = dict(a=addr(0), a_scale=addr(1), w=addr(2), w_scale=addr(6))
    for k, v in kw.items():
        (d if k in d else p)[k] = v
    dims = qz.MatmulDims(**d)
    for i, c in enumerate(out_cols):
        dims.out_cols[i] = c
        dims.out_stride[i] = (out_stride or out_cols)[i]
    ptrs = (ctypes.c_void_p * 8)(*[addr(o) if isinstance(o, int) and o < 64 else o for o in outs])
    return L.gdr_matmul_i8(ctypes.addressof(dims), p["a"], p["a_scale"], p["w"], p["w_scale"], bias,
                           None if null_outs else ctypes.addressof(ptrs), None)


def test_matmul_refusals(L):
    assert L.gdr_matmul_i8(*[None] * 8) == ENULL
    for name in ("a", "a_scale", "w", "w_scale"):
        assert product(L, **{name: None}) == ENULL, name
    assert product(L, null_outs=True) == ENULL
    assert product(L, outs=(4, None)) == ENULL
    for kw in (dict(M=-1), dict(K=0), dict(K=131072, a_stride=131072, w_stride=131072), dict(n_out=0), dict(n_out=9),
               dict(a_stride=-1), dict(w_stride=-1), dict(out_cols=(0, 16)), dict(out_stride=(31, 16)),
               dict(out_cols=((1 << 30), 16)), dict(M=2147483647, out_cols=(1 << 20, 1 << 20)),
               dict(M=1 << 30, a_stride=1 << 40), dict(M=(1 << 30) + 1)):
        assert product(L, **kw) == ESHAPE, kw
    assert product(L, out_dtype=2) == EUNSUP
    for kw in (dict(a_scale=addr(1, 2)), dict(w_scale=addr(6, 1)), dict(bias=addr(3, 2)), dict(outs=(addr(4, 1), 5)),
               dict(out_dtype=1, outs=(addr(4, 2), 5))):
        assert product(L, **kw) == EALIGN, kw
    for kw in (dict(outs=(0, 5)), dict(outs=(1, 5)), dict(outs=(2, 5)), dict(outs=(4, 3)), dict(outs=(6, 5)), dict(outs=(4, 4)),
               # column ranges of one array, one column too near
               dict(outs=(addr(4), addr(4, 62)), out_stride=(48, 48)),
               # and with unequal rows
               dict(outs=(addr(4), addr(4, 64)), out_stride=(48, 50)),
               # and wrapping into the next row
               dict(outs=(addr(4), addr(4, 66)), out_stride=(48, 48))):
        assert product(L, **kw) == EALIAS, kw
    assert product(L, M=0, a=None, a_scale=None, w=None, w_scale=None, null_outs=True, bias=None) == OK


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i8(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


GOOD_NORM = dict(x=bf(2, 3, 64), weight=bf(64), residual=bf(2, 3, 64))


@pytest.mark.parametrize("kw,error,match", [
    (dict(weight=bf(65)), ValueError, "weight must be"),
    (dict(weight=torch.zeros(64, dtype=torch.float64)), TypeError, "weight must be"),
    (dict(weight=bf(128)[::2]), ValueError, "weight must be contiguous"),
    (dict(x=torch.zeros(2, 3, 64), residual=torch.zeros(2, 3, 64)), TypeError, "weight must be"),
    (dict(x=torch.zeros(2, 3, 64, dtype=torch.float16)), TypeError, "x must be"),
    (dict(residual=bf(2, 2, 64)), ValueError, "residual must be"),
    (dict(residual=torch.zeros(2, 3, 64)), TypeError, "residual must be"),
    (dict(residual=None, out_residual=bf(2, 3, 64)), ValueError, "without a residual"),
    (dict(out_residual=bf(2, 3, 65)), ValueError, "out_residual must be"),
    (dict(out_residual=torch.zeros(2, 3, 64)), TypeError, "out_residual must be"),
    (dict(x=bf(2, 64, 3).transpose(1, 2)), ValueError, "values of a row"),
    (dict(x=bf(2, 4, 64)[:, :3]), ValueError, "evenly spaced"),
    (dict(q=i8(6, 64)), ValueError, "q must be"),
    (dict(q=bf(2, 3, 64)), TypeError, "q must be"),
    (dict(scale=torch.zeros(3, 2)), ValueError, "scale must be"),
    (dict(eps=-1e-6), ValueError, "eps must be"),
    (dict(eps=float("nan")), ValueError, "eps must be"),
    (dict(x=bf(2, 0), residual=None, weight=bf(0)), ValueError, "x must be"),
    (dict(x=bf(1, 32769), residual=None, weight=bf(32769)), ValueError, "at most"),
    (dict(), ValueError, "GPU tensor"),
])
def test_add_rmsnorm_binding_refusals(kw, error, match):
    with pytest.raises(error, match=match):
        gdr.add_rmsnorm_i8(**{**GOOD_NORM, **kw})


@pytest.mark.parametrize("kw,error,match", [
    (dict(o=bf(2, 4, 48), gate=bf(2, 4, 48), weight=bf(48)), ValueError, "dv must be"),
    (dict(gate=bf(2, 3, 64)), ValueError, "gate must be"),
    (dict(gate=torch.zeros(2, 4, 64, dtype=torch.int8)), TypeError, "gate must be"),
    (dict(weight=bf(4, 64)), ValueError, "weight must be"),
    (dict(o=bf(2, 8, 64)[:, ::2]), ValueError, "values of a row"),
    (dict(o=bf(1, 513, 64), gate=bf(1, 513, 64)), ValueError, "HV"),
    (dict(q=i8(2, 4, 64)), ValueError, "q must be"),
    (dict(), ValueError, "GPU tensor"),
])
def test_gated_rmsnorm_binding_refusals(kw, error, match):
    good = dict(o=bf(2, 4, 64), gate=bf(2, 4, 64), weight=bf(64))
    with pytest.raises(error, match=match):
        gdr.gated_rmsnorm_i8(**{**good, **kw})


@pytest.mark.parametrize("kw,error,match", [
    (dict(w=i8(12, 31)), ValueError, "a must be"),
    (dict(w=bf(12, 32)), TypeError, "w must be int8"),
    (dict(a=torch.zeros(5, 32, dtype=torch.uint8)), TypeError, "a must be int8"),
    (dict(a_scale=torch.zeros(4)), ValueError, "a_scale must be"),
    (dict(a_scale=None), TypeError, "a_scale is required"),
    (dict(w_scale=torch.zeros(12, dtype=torch.bfloat16)), TypeError, "w_scale must be"),
    (dict(w_scale=torch.zeros(24)[::2]), ValueError, "w_scale must be contiguous"),
    (dict(bias=torch.zeros(11)), ValueError, "bias must be"),
    (dict(out=(6, 7)), ValueError, "add up"),
    (dict(out=(12, 0)), ValueError, "add up"),
    (dict(out=()), ValueError, "1 to 8"),
    (dict(out=(1,) * 9), ValueError, "1 to 8"),
    (dict(out_dtype=torch.float16), TypeError, "out must be"),
    (dict(out=bf(4, 12)), ValueError, "out must be"),
    (dict(out=(bf(5, 6), torch.zeros(5, 6))), TypeError, "one type"),
    (dict(a=i8(5, 64)[:, ::2]), ValueError, "values of a row"),
    (dict(w=i8(0, 32), w_scale=torch.zeros(0)), ValueError, "N must be"),
    (dict(a=i8(5, 0), w=i8(12, 0)), ValueError, "K in 1"),
    (dict(), ValueError, "GPU tensor"),
])
def test_matmul_binding_refusals(kw, error, match):
    good = dict(a=i8(5, 32), a_scale=torch.zeros(5), w=i8(12, 32), w_scale=torch.zeros(12))
    with pytest.raises(error, match=match):
        gdr.matmul_i8(**{**good, **kw})


def test_quantize_rows():
    w = torch.tensor([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [2.54, -1.27, 0.01, 0.0]])
    q, s = gdr.quantize_rows_i8(w)
    assert q.tolist()[:2] == [[127, -64, 0, 2], [0, 0, 0, 0]] and s.tolist()[:2] == [1.0, 0.0]
    err = (q.double() * s.double()[:, None] - w.double()).abs().amax(1)
    assert bool((err <= s.double() * 0.5 * (1 + 2.0 ** -20)).all())
    with pytest.raises(ValueError, match="matrix"):
        gdr.quantize_rows_i8(torch.zeros(4))

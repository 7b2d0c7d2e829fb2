"""Refusals of the operators before and beside the recurrence, on the host: the C entry points with
fake device addresses (only on calls whose validation fails, or that have nothing to do), and the Python
binding with CPU tensors, whose checks of shapes and types run before the device is looked at."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gated_delta_rule_70_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdr_layer.h")
OK, ENULL, ESHAPE, EUNSUP, EALIGN, EALIAS, EWS = range(7)
BASE, SLOT = 1 << 40, 1 << 34
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


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
    assert names == {"gdr_causal_conv", "gdr_qk_norm_rope", "gdr_selective_scan", "gdr_selective_scan_step"}
    out = subprocess.run(["nm", "-D", "--defined-only", gdr.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT\s+(\w+)$", out, re.M))


def test_limits_match_the_header():
    src = open(HEADER).read()
    for name, value in (("GDR_CONV_MAX_OUT", layer.CONV_MAX_OUT), ("GDR_SCAN_MAX_STATES", layer.SCAN_MAX_STATES),
                        ("GDR_QK_MAX_DIM", layer.QK_MAX_DIM)):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == value
    assert layer.MAX_ROWS == 1 << 30 and layer.MAX_CHANNELS == 1 << 24 and layer.MAX_SEQS == gdr.VARLEN_MAX_SEQS


def split(kw, d):
    p = {}
    for k, v in kw.items():
        (d if k in d else p)[k] = v
    return p


def conv(L, **kw):
    d = dict(B=2, T=5, D=64, W=4, dtype=0, weight_dtype=0, flags=1, n_out=2, out_cols=(24, 40), out_stride=(24, 40), x_stride=64)
    p = dict(cu=None, x=addr(0), w=addr(1), bias=addr(2), state=addr(3), end=addr(4), outs=(addr(5), addr(6)))
    p.update(split(kw, d))
    d["out_cols"] = (ctypes.c_int32 * 8)(*d["out_cols"])
    d["out_stride"] = (ctypes.c_int64 * 8)(*d["out_stride"])
    dims = layer.ConvDims(**d)
    outs = None if p["outs"] is None else (ctypes.c_void_p * 8)(*p["outs"])
    return L.gdr_causal_conv(ctypes.addressof(dims), p["cu"], p["x"], p["w"], p["bias"], p["state"],
                             None if outs is None else ctypes.addressof(outs), p["end"], None)


@pytest.mark.parametrize("want,kw", [
    (ESHAPE, dict(B=-1)), (ESHAPE, dict(T=-1)), (ESHAPE, dict(B=1 << 16, T=1 << 15)), (ESHAPE, dict(D=0)),
    (ESHAPE, dict(D=(1 << 24) + 1)), (ESHAPE, dict(W=0)), (EUNSUP, dict(W=1)), (EUNSUP, dict(W=5)), (EUNSUP, dict(dtype=2)),
    (EUNSUP, dict(dtype=1, weight_dtype=0)), (EUNSUP, dict(weight_dtype=2)), (EUNSUP, dict(flags=2)), (ESHAPE, dict(n_out=0)),
    (ESHAPE, dict(n_out=9)), (ESHAPE, dict(out_cols=(24, 39))), (ESHAPE, dict(out_cols=(24, 41))), (ESHAPE, dict(out_cols=(64, 0))),
    (ESHAPE, dict(out_stride=(23, 40))), (ESHAPE, dict(x_stride=-1)), (ESHAPE, dict(x_stride=1 << 61)),
    (ENULL, dict(x=None)), (ENULL, dict(w=None)), (ENULL, dict(outs=None)), (ENULL, dict(outs=(addr(5), None))),
    (EALIGN, dict(x=addr(0, 1))), (EALIGN, dict(state=addr(3, 1))), (EALIGN, dict(outs=(addr(5), addr(6, 1)))),
    (EALIGN, dict(end=addr(4, 1))), (EALIGN, dict(cu=addr(7, 2))), (EALIGN, dict(weight_dtype=1, w=addr(1, 2))),
    (ESHAPE, dict(cu=addr(7), B=0)), (ESHAPE, dict(cu=addr(7), B=4097)),
    (EALIAS, dict(outs=(addr(0), addr(6)))), (EALIAS, dict(outs=(addr(5), addr(5, 24)))), (EALIAS, dict(end=addr(3, 2))),
    (EALIAS, dict(end=addr(0))), (EALIAS, dict(end=addr(5))), (EALIAS, dict(outs=(addr(5), addr(3)))),
    (EALIAS, dict(cu=addr(7), outs=(addr(7), addr(6)))), (EALIAS, dict(cu=addr(7), end=addr(7))),
    (OK, dict(B=0)), (OK, dict(B=0, x=None, w=None, outs=None, end=None)), (OK, dict(T=0, end=None)),
])
def test_conv_refusals(L, want, kw):
    assert conv(L, **kw) == want
    assert L.gdr_causal_conv(None, *[None] * 8) == ENULL


def qk(L, **kw):
    d = dict(rows=5, q_heads=4, k_heads=2, dim=64, rotated=32, table_rows=100, period=5, position_bits=32, dtype=0, weight_dtype=0,
             flags=0, eps=1e-6, q_stride=256, k_stride=128, out_q_stride=256, out_k_stride=128)
    p = dict(q=addr(0), k=addr(1), qw=addr(2), kw=addr(3), cos=addr(4), sin=addr(5), pos=None, oq=addr(6), ok=addr(7))
    p.update(split(kw, d))
    dims = layer.QkDims(**d)
    return L.gdr_qk_norm_rope(ctypes.addressof(dims), *[p[n] for n in ("q", "k", "qw", "kw", "cos", "sin", "pos", "oq", "ok")], None)


@pytest.mark.parametrize("want,kw", [
    (ESHAPE, dict(rows=-1)), (ESHAPE, dict(rows=(1 << 30) + 1)), (ESHAPE, dict(q_heads=0)), (ESHAPE, dict(k_heads=65537)),
    (ESHAPE, dict(dim=0)), (EUNSUP, dict(dim=513)), (ESHAPE, dict(rotated=33)), (ESHAPE, dict(rotated=66)), (ESHAPE, dict(rotated=-2)),
    (ESHAPE, dict(table_rows=0)), (ESHAPE, dict(period=0)), (EUNSUP, dict(pos=addr(8), position_bits=16)), (EUNSUP, dict(dtype=2)),
    (EUNSUP, dict(dtype=1)), (EUNSUP, dict(flags=2)), (EUNSUP, dict(eps=-1.0)), (EUNSUP, dict(eps=float("nan"))),
    (EUNSUP, dict(eps=float("inf"))), (ESHAPE, dict(q_stride=-1)), (ESHAPE, dict(out_q_stride=255)), (ESHAPE, dict(out_k_stride=127)),
    (ENULL, dict(q=None)), (ENULL, dict(k=None)), (ENULL, dict(cos=None)), (ENULL, dict(sin=None)), (ENULL, dict(oq=None)),
    (ENULL, dict(ok=None)), (EALIGN, dict(q=addr(0, 1))), (EALIGN, dict(cos=addr(4, 2))), (EALIGN, dict(pos=addr(8, 2))),
    (EALIGN, dict(pos=addr(8, 4), position_bits=64)), (EALIAS, dict(oq=addr(1))), (EALIAS, dict(ok=addr(0))), (EALIAS, dict(ok=addr(6))),
    (EALIAS, dict(oq=addr(0, 2))), (EALIAS, dict(oq=addr(0), q_stride=300)), (EALIAS, dict(oq=addr(4))), (EALIAS, dict(ok=addr(3))),
    (EALIAS, dict(pos=addr(8), oq=addr(8))), (OK, dict(rows=0)), (OK, dict(rows=0, q=None, k=None, oq=None, ok=None)),
])
def test_qk_refusals(L, want, kw):
    assert qk(L, **kw) == want
    assert L.gdr_qk_norm_rope(None, *[None] * 10) == ENULL


def scan(L, step=False, **kw):
    d = dict(B=2, T=1 if step else 5, D=64, N=16, G=2, dtype=0, dt_dtype=0, flags=1, x_stride=64, dt_stride=64, z_stride=64, b_stride=32,
             c_stride=32, out_stride=64)
    p = dict(cu=None, x=addr(0), dt=addr(1), A=addr(2), B_=addr(3), C=addr(4), skip=addr(5), z=addr(6), bias=addr(7), h0=addr(8),
             out=addr(9), ht=addr(10), ws=None, ws_bytes=0)
    p.update(split(kw, d))
    dims = layer.ScanDims(**d)
    rest = [p[n] for n in ("x", "dt", "A", "B_", "C", "skip", "z", "bias", "h0", "out", "ht")]
    if step:
        return L.gdr_selective_scan_step(ctypes.addressof(dims), *rest, None)
    return L.gdr_selective_scan(ctypes.addressof(dims), p["cu"], *rest, p["ws"], p["ws_bytes"], None)


BOTH = [
    (ESHAPE, dict(B=-1)), (ESHAPE, dict(T=-1)), (ESHAPE, dict(D=0)), (ESHAPE, dict(D=1 << 25)), (ESHAPE, dict(N=0)),
    (EUNSUP, dict(N=129)), (ESHAPE, dict(G=0)), (ESHAPE, dict(G=3)), (EUNSUP, dict(dtype=2)), (EUNSUP, dict(dtype=1, dt_dtype=0)),
    (EUNSUP, dict(dt_dtype=2)), (EUNSUP, dict(flags=2)), (ESHAPE, dict(x_stride=-1)), (ESHAPE, dict(b_stride=-1)),
    (ESHAPE, dict(z_stride=-1)), (ESHAPE, dict(out_stride=63)), (ESHAPE, dict(c_stride=1 << 62)),
    (ENULL, dict(x=None)), (ENULL, dict(dt=None)), (ENULL, dict(A=None)), (ENULL, dict(B_=None)), (ENULL, dict(C=None)),
    (ENULL, dict(out=None)), (EALIGN, dict(x=addr(0, 1))), (EALIGN, dict(A=addr(2, 2))), (EALIGN, dict(h0=addr(8, 2))),
    (EALIGN, dict(dt_dtype=1, dt=addr(1, 2))), (EALIAS, dict(out=addr(0))), (EALIAS, dict(out=addr(6))), (EALIAS, dict(ht=addr(8, 4))),
    (EALIAS, dict(ht=addr(9))), (EALIAS, dict(out=addr(8))), (EALIAS, dict(ht=addr(2))), (OK, dict(B=0)),
]


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("want,kw", BOTH)
def test_scan_refusals(L, step, want, kw):
    assert scan(L, step, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (ESHAPE, dict(B=1 << 16, T=1 << 15)), (ESHAPE, dict(cu=addr(11), B=0)), (ESHAPE, dict(cu=addr(11), B=4097)),
    (EALIGN, dict(cu=addr(11, 2))), (EALIAS, dict(cu=addr(11), ht=addr(11))), (OK, dict(T=0, ht=None)),
    (OK, dict(T=0, ht=None, x=None, dt=None, A=None, B_=None, C=None, out=None)),
])
def test_prompt_scan_refusals(L, want, kw):
    assert scan(L, **kw) == want
    assert L.gdr_selective_scan(None, *[None] * 13, 0, None) == ENULL


LONG = dict(B=1, T=4096, N=16, D=64, G=1, b_stride=16, c_stride=16)


@pytest.mark.parametrize("want,kw", [
    (EWS, dict(ws=None)), (EWS, dict(ws=addr(12), ws_bytes=-1)), (EALIGN, dict(ws=addr(12, 2))), (EALIAS, dict(ws=addr(0))),
    (EALIAS, dict(ws=addr(9))), (EALIAS, dict(ws=addr(8))), (EALIAS, dict(ws=addr(10))),
])
def test_scan_workspace_refusals(L, want, kw):
    need = gdr.selective_scan_workspace_bytes(1, 4096, 64, 16)
    assert need > 0
    kw = {"ws_bytes": need, **kw}
    if kw["ws_bytes"] < 0:
        kw["ws_bytes"] += need
    assert scan(L, **LONG, **kw) == want


def test_scan_workspace():
    """Only where channels are few and sequences long; what is needed never passes what the entries of
    cu_seqlens could ask for."""
    size = gdr.selective_scan_workspace_bytes
    assert size(1, 4097, 4096, 16) == 0 and size(8, 512, 4096, 16) == 0 and size(1, 64, 64, 16) == 0
    assert size(0, 100, 64, 16) == 0 and size(1, 100, 63, 16, groups=2) == 0 and size(1, 4096, 64, 129) == 0
    for B, T, D, N, G, packed in ((1, 4096, 64, 16, 1, False), (2, 100000, 300, 5, 3, False), (4, 8192, 128, 16, 1, True)):
        n = size(B, T, D, N, groups=G, packed=packed)
        assert n > 0 and n % (4 * B * D * (N + 1)) == 0
        segs = n // (4 * B * D * (N + 1))
        assert 2 <= segs <= T // 64 + 1
    assert size(4096, 1 << 20, 64, 16, packed=True) == 0


@pytest.mark.parametrize("T", [0, 2])
def test_step_takes_one_token(L, T):
    assert scan(L, True, T=T) == ESHAPE
    assert L.gdr_selective_scan_step(None, *[None] * 12) == ENULL


# ---- the Python binding ----------------------------------------------------------------------

def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def py_conv(**kw):
    a = dict(x=z(2, 5, 64), weight=z(64, 4), bias=z(64), state=z(2, 3, 64))
    a.update(kw)
    return gdr.causal_conv(**a)


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU tensor", {}), (ValueError, r"\[B, T, D\]", dict(x=z(5, 64))), (ValueError, "channels", dict(x=z(2, 5, 0))),
    (TypeError, "bfloat16 or float32", dict(x=z(2, 5, 64, dtype=torch.float16))), (ValueError, "weight", dict(weight=z(64, 5))),
    (ValueError, "weight", dict(weight=z(63, 4))), (TypeError, "weight", dict(weight=z(64, 4, dtype=torch.float64))),
    (ValueError, "weight must be contiguous", dict(weight=z(4, 64).t())), (TypeError, "bias", dict(bias=z(64, dtype=F32))),
    (ValueError, "bias", dict(bias=z(63))), (ValueError, "activation", dict(activation="gelu")), (ValueError, "state", dict(state=z(2, 4, 64))),
    (TypeError, "state", dict(state=z(2, 3, 64, dtype=F32))), (ValueError, "out_state", dict(out_state=z(1, 3, 64))),
    (ValueError, "channels", dict(out=(32, 31))), (ValueError, "channels", dict(out=(64, 0))), (ValueError, "1 to 8", dict(out=())),
    (ValueError, "1 to 8", dict(out=(8,) * 9)), (ValueError, "out must be", dict(out=z(2, 4, 64))), (TypeError, "out", dict(out=z(2, 5, 64, dtype=F32))),
    (ValueError, "evenly", dict(x=z(2, 9, 64)[:, :5])), (ValueError, "contiguous", dict(x=z(2, 5, 128)[..., ::2])),
    (ValueError, "packed", dict(cu_seqlens=z(3, dtype=I32))), (ValueError, "cu_seqlens", dict(x=z(5, 64), cu_seqlens=z(1, dtype=I32))),
    (TypeError, "cu_seqlens", dict(x=z(5, 64), cu_seqlens=z(3, dtype=torch.int64))),
    (ValueError, "cu_seqlens", dict(x=z(5, 64), cu_seqlens=z(4098, dtype=I32))),
    (ValueError, "cu_seqlens", dict(x=z(5, 64), cu_seqlens=z(6, dtype=I32)[::2])), (ValueError, "state", dict(x=z(5, 64), cu_seqlens=z(4, dtype=I32))),
    (ValueError, "GPU tensor", dict(x=z(5, 64), cu_seqlens=z(3, dtype=I32))), (ValueError, "GPU tensor", dict(x=z(1, 5, 64), cu_seqlens=z(3, dtype=I32))),
])
def test_python_conv(error, match, kw):
    with pytest.raises(error, match=match):
        py_conv(**kw)


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, r"\[B, D\]", dict(x=z(2, 1, 64))), (ValueError, "state", dict(state=z(3, 3, 64))), (ValueError, "GPU tensor", {}),
])
def test_python_conv_step(error, match, kw):
    with pytest.raises(error, match=match):
        gdr.causal_conv_step(**{**dict(x=z(2, 64), weight=z(64, 4), state=z(2, 3, 64)), **kw})


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU tensor", {}), (ValueError, "HQ", dict(k=z(5, 2, 32))), (ValueError, "HQ", dict(k=z(4, 2, 64))),
    (ValueError, "512", dict(q=z(5, 4, 514), k=z(5, 2, 514))), (TypeError, "k must be", dict(k=z(5, 2, 64, dtype=F32))),
    (TypeError, "bfloat16 or float32", dict(q=z(5, 4, 64, dtype=torch.float16))), (ValueError, "q_weight", dict(q_weight=z(63))),
    (TypeError, "k_weight", dict(k_weight=z(64, dtype=F32))), (TypeError, "together", dict(cos=None)), (ValueError, "cos", dict(cos=z(9, 33, dtype=F32))),
    (ValueError, "sin", dict(sin=z(8, 16, dtype=F32))), (TypeError, "sin", dict(sin=z(9, 16))), (TypeError, "positions", dict(positions=z(5, dtype=torch.int16))),
    (ValueError, "positions", dict(positions=z(4, dtype=I32))), (TypeError, "without cos", dict(cos=None, sin=None, positions=z(5, dtype=I32))),
    (ValueError, "out_q", dict(out_q=z(5, 2, 64))), (TypeError, "out_k", dict(out_k=z(5, 2, 64, dtype=F32))), (ValueError, "eps", dict(eps=-1.0)),
    (ValueError, "eps", dict(eps=1e39)), (ValueError, "contiguous", dict(q=z(5, 4, 128)[..., :64])),
])
def test_python_qk(error, match, kw):
    a = dict(q=z(5, 4, 64), k=z(5, 2, 64), q_weight=z(64), k_weight=z(64), cos=z(9, 16, dtype=F32), sin=z(9, 16, dtype=F32))
    with pytest.raises(error, match=match):
        gdr.qk_norm_rope(**{**a, **kw})


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU tensor", {}), (ValueError, r"\[B, T, D\]", dict(x=z(5, 64))), (ValueError, "A must", dict(A=z(64, 129, dtype=F32))),
    (ValueError, "A must", dict(A=z(63, 16, dtype=F32))), (TypeError, "A must", dict(A=z(64, 16))), (ValueError, "dt", dict(dt=z(2, 4, 64))),
    (TypeError, "dt", dict(dt=z(2, 5, 64, dtype=torch.float16))), (ValueError, "B must", dict(B=z(2, 5, 15))), (ValueError, "C must", dict(C=z(2, 5, 1, 16))),
    (ValueError, "groups", dict(B=z(2, 5, 3, 16))), (TypeError, "C must", dict(C=z(2, 5, 16, dtype=F32))), (ValueError, "z must", dict(z=z(2, 5, 63))),
    (TypeError, "D must", dict(D=z(64))), (ValueError, "dt_bias", dict(dt_bias=z(63, dtype=F32))), (ValueError, "h0", dict(h0=z(2, 64, 15, dtype=F32))),
    (TypeError, "h0", dict(h0=z(2, 64, 16))), (ValueError, "out", dict(out=z(2, 5, 63))), (ValueError, "ht", dict(ht=z(1, 64, 16, dtype=F32))),
])
def test_python_scan(error, match, kw):
    a = dict(x=z(2, 5, 64), dt=z(2, 5, 64), A=z(64, 16, dtype=F32), B=z(2, 5, 16), C=z(2, 5, 16))
    with pytest.raises(error, match=match):
        gdr.selective_scan(**{**a, **kw})


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "GPU tensor", {}), (ValueError, r"\[B, D\]", dict(x=z(2, 1, 64))), (ValueError, "h0", dict(state=z(3, 64, 16, dtype=F32))),
    (ValueError, "B must", dict(B=z(3, 16))),
])
def test_python_scan_step(error, match, kw):
    a = dict(x=z(2, 64), dt=z(2, 64), A=z(64, 16, dtype=F32), B=z(2, 16), C=z(2, 16), state=z(2, 64, 16, dtype=F32))
    with pytest.raises(error, match=match):
        gdr.selective_scan_step(**{**a, **kw})


def test_rope_table():
    cos, sin = gdr.rope_table(70000, 6, base=100.0)
    assert cos.shape == sin.shape == (70000, 3) and cos.dtype == F32
    for p, i in ((0, 0), (1, 2), (69999, 0), (69999, 1)):
        angle = torch.tensor(p * 100.0 ** (-2 * i / 6), dtype=torch.float64)
        assert abs(cos[p, i].double() - angle.cos()) < 2e-7 and abs(sin[p, i].double() - angle.sin()) < 2e-7
    for bad in (dict(length=0, rotated=6), dict(length=3, rotated=5), dict(length=3, rotated=0)):
        with pytest.raises(ValueError):
            gdr.rope_table(**bad)


def test_bound_arguments_match_the_header(L):
    """As many of them as the header declares: one more would be passed as a C int, a stream's handle cut."""
    for name, args in re.findall(r"^\s*int\s+(gdr_\w+)\s*\(([^)]*)\)", open(HEADER).read(), re.M):
        assert len(getattr(L, name).argtypes) == args.count(",") + 1, name

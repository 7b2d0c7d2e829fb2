"""matmul_i8 on every one of its forms (i8_forms.py says which sizes run which, and test_i8_plan.py
that they do).  Tolerance: the int32 sum is exact; its conversion and two scales round three times,
the bias's addition once more, a bf16 output once to half a step, 2^-8."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gpu_util import note
from i8_forms import FORMS, TWO, name

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def operand(rows, K, pad, off, seed):
    """Codes in an array that ends with their last byte."""
    gen = torch.Generator("cuda").manual_seed(seed)
    flat = torch.randint(-128, 128, ((rows - 1) * (K + pad) + K + off,), device="cuda", dtype=torch.int8, generator=gen)
    return flat[off:].as_strided((rows, K), (K + pad, 1))


def product(M, N, K, pad=0, off=0):
    a, w = operand(M, K, pad, off, 1), operand(N, K, pad, off, 2)
    gen = torch.Generator("cuda").manual_seed(3)
    sa, sw = (torch.rand(n, device="cuda", generator=gen) + 0.1 for n in (M, N))
    bias = torch.randn(N, device="cuda", generator=gen) * K ** 0.5 * 1000
    size = (a.double() @ w.double().t()).mul_(sa.double()[:, None]).mul_(sw.double())
    return a, sa, w, sw, bias, size


def check(y, size, bias):
    """y [M, N] against the product in 64 bits without bias (and the bias, or None)."""
    ref = size if bias is None else size + bias.double()
    tol = size.abs().mul_(3 * U)
    if bias is not None:
        tol.add_((ref.abs() + tol) * U)
    tol.mul_(1 + 4 * U)          # the roundings' products
    if y.dtype == BF:
        tol.add_((ref.abs() + tol) * 2.0 ** -8)
    off = (y.double() - ref).abs_()
    assert bool((off <= tol).all()), f"{float((off / tol).nan_to_num(0).max())} times the tolerance"


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", FORMS, ids=name)
def test_form(case, dtype):
    form, moved, M, N, K, pad, off = case
    a, sa, w, sw, bias, size = product(M, N, K, pad, off)
    room = torch.full((M + 2, N), 7.0, dtype=dtype, device="cuda")
    b = bias if dtype == F32 else None
    note(f"{name(case)} {dtype}")
    gdr.matmul_i8(a, sa, w, sw, bias=b, out=room[1:M + 1])
    check(room[1:M + 1], size, b)
    assert bool((room[0] == 7.0).all()) and bool((room[M + 1] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [t[:3] for t in TWO])
def test_two_launches(M, N, K, dtype):
    a, sa, w, sw, bias, size = product(M, N, K)
    room = torch.full((M + 2, N), 7.0, dtype=dtype, device="cuda")
    b = bias if dtype == F32 else None
    note(f"two launches {M}x{N}x{K} {dtype}")
    gdr.matmul_i8(a, sa, w, sw, bias=b, out=room[1:M + 1])
    check(room[1:M + 1], size, b)
    assert bool((room[0] == 7.0).all()) and bool((room[M + 1] == 7.0).all())


def splits(N):
    """Ways to cut N columns: outputs of a layer, many of them inside one store of 4 or 8 columns at
    the first column, in the middle and at the last one."""
    third = N // 3 // 16 * 16
    half = N // 2 | 1
    return {"layer": (third, third, N - 2 * third),
            "front": (3, 1, 1, 2, half, 1, 2, N - half - 10),
            "back": (N - 18, 5, 1, 7, 2, 1, 1, 1),
            "odd": (half - 6, N - half - 7, 13)}


def check_splits(M, N, size, bias, dtype, call):
    for way, cols in splits(N).items():
        # side by side in one array that is written nowhere else, three columns apart
        room = torch.full((M + 2, N + 3 * len(cols) + 2), 7.0, dtype=dtype, device="cuda")
        at, parts = 1, []
        for n in cols:
            parts.append(room[1:M + 1, at:at + n])
            at += n + 3
        note(f"outputs {way} {M}x{N} {dtype}")
        call(parts)
        check(torch.cat(parts, 1), size, bias)
        for p in parts:
            p.fill_(7.0)
        assert bool((room == 7.0).all()), way
        # each dense, at the end of an array of its own
        own = [torch.full((M * n + 5,), 7.0, dtype=dtype, device="cuda") for n in cols]
        call([t[5:].view(M, n) for t, n in zip(own, cols)])
        check(torch.cat([t[5:].view(M, n) for t, n in zip(own, cols)], 1), size, bias)
        assert all(bool((t[:5] == 7.0).all()) for t in own), way


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", FORMS, ids=name)
def test_outputs_that_end_inside_a_store(case, dtype):
    form, moved, M, N, K, pad, off = case
    a, sa, w, sw, bias, size = product(M, N, K, pad, off)
    b = bias if dtype == F32 else None
    check_splits(M, N, size, b, dtype, lambda out: gdr.matmul_i8(a, sa, w, sw, bias=b, out=out))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [t[:3] for t in TWO])
def test_outputs_of_two_launches(M, N, K, dtype):
    a, sa, w, sw, bias, size = product(M, N, K)
    b = bias if dtype == F32 else None
    check_splits(M, N, size, b, dtype, lambda out: gdr.matmul_i8(a, sa, w, sw, bias=b, out=out))

"""add_rmsnorm_i8 on rows whose products of value and weight lie below fp32's normal range.

Codes are those of the exact quotient and are compared exactly; the scale is rounded once from
fp64: 1.01 U relative, and half a step of fp32's smallest numbers, 2^-150, where it is one of those."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gpu_util import note

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def reference(x, w, r, eps):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    t = s.double() * w.double()
    top = t.abs().amax(-1)
    q = torch.round(t * 127.0 / torch.where(top > 0, top, 1.0)[:, None])
    return s, q, torch.where(top > 0, top / torch.sqrt(s.double().square().mean(-1) + eps) / 127.0, 0.0)


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("D", [1, 96, 333, 1000, 2048, 4096, 4097, 8192, 16384, 32768])
def test_products_below_the_normal_range(D, types):
    rows = [(1e-30, 1e-13), (1e-30, 1e-8), (1e-20, 1e-18), (1e-30, 1e-20), (1e-38, 1e-38), (3.0, 1e-38), (1e-38, 3.0)]
    for i, (size, weight) in enumerate(rows):
        x, r = ((size * rand(4, D, seed=10 * i + j)).to(types[0]) for j in (1, 2))
        w = (weight * rand(D, seed=10 * i + 3)).to(types[1])
        x[2] = r[2] = 0.0           # a padding row among them
        x[3], r[3] = rand(D, seed=4).to(types[0]), rand(D, seed=5).to(types[0])
        for res, eps in ((None, 1e-6), (r, 0.0)):
            s, q_ref, scale_ref = reference(x, w, res, eps)
            note(f"D={D} {types} values {size} weights {weight} residual={res is not None}")
            stream = None if res is None else res.cuda()
            q, scale, out = gdr.add_rmsnorm_i8(x.cuda(), w.cuda(), residual=stream, out_residual=stream, eps=eps)
            assert torch.equal(q.cpu().double(), q_ref)
            assert bool(((scale.cpu().double() - scale_ref).abs() <= 1.01 * U * scale_ref + 2.0 ** -150).all())
            assert out is stream and (res is None or torch.equal(out.cpu(), s))


def test_one_wave_a_row():
    """The form for many short rows, with rows of either kind next to each other."""
    M, D = 5000, 1000
    x = rand(M, D, seed=1) * torch.where(torch.arange(M) % 3 == 0, 1e-30, 1.0)[:, None]
    x, w = x.to(BF), (1e-13 * rand(D, seed=2)).to(BF)
    s, q_ref, scale_ref = reference(x, w, None, 0.0)
    note("one wave a row")
    q, scale, _ = gdr.add_rmsnorm_i8(x.cuda(), w.cuda(), eps=0.0)
    assert torch.equal(q.cpu().double(), q_ref)
    assert bool(((scale.cpu().double() - scale_ref).abs() <= 1.01 * U * scale_ref + 2.0 ** -150).all())

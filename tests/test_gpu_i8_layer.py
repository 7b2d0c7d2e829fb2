"""The 8-bit operators together with the delta rule, as a layer (examples/int8_layer.py), against
the same layer written plainly: dequantised weights, codes from the definitions in 64 bits, the
fp64 oracle for the recurrence.

Tolerance: the delta rule is held to TOL = 2e-3 of its largest output, a quarter of a step of
the int8 codes that follow, so up to a quarter of the codes may be a neighbour's: an error of
at most half a step in the 2-norm, where a row's values are about a tenth of its largest:
0.5 / 12.7 = 0.04, and bf16 outputs on top, 0.004."""
import importlib.util
import os

import pytest
import torch

import gated_delta_rule_70_amd as gdr
import oracle
from gpu_util import note

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("int8_layer", os.path.join(ROOT, "examples", "int8_layer.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def codes(t):
    top = t.abs().amax(-1, keepdim=True)
    return torch.round(t * 127.0 / top) * (top / 127.0)


def plain(layer, x, stream, state):
    c = lambda t: t.detach().double().cpu()  # noqa: E731
    B, T, _ = x.shape
    HK, HV, dk, dv = layer.HK, layer.HV, layer.dk, layer.dv
    s = (x.float() + stream.float()).bfloat16()
    n = c(s) * c(layer.norm) * torch.rsqrt(c(s).square().mean(-1, keepdim=True) + 1e-6)
    n = codes(n)
    p = (n @ (c(layer.w_in) * c(layer.w_in_scale)[:, None]).t()).bfloat16()
    q, k, v, z = p.split((HK * dk, HK * dk, HV * dv, HV * dv), -1)
    g = n @ (c(layer.w_gate) * c(layer.w_gate_scale)[:, None]).t() + c(layer.gate_bias)
    a, b = g.split((HV * dk, HV), -1)
    k = torch.nn.functional.normalize(k.double().view(B, T, HK, dk), dim=-1, eps=1e-12)
    o, ht = oracle.sequential(q=q.double().view(B, T, HK, dk), k=k, v=v.double().view(B, T, HV, dv),
                              g=-torch.nn.functional.softplus(a.view(B, T, HV, dk)), beta=torch.sigmoid(b), h0=c(state))
    o = torch.from_numpy(o)
    z = z.double().view(B, T, HV, dv)
    n = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) * c(layer.head_norm) * z * torch.sigmoid(z)
    y = codes(n.flatten(-2)) @ (c(layer.w_out) * c(layer.w_out_scale)[:, None]).t()
    return y, s, torch.from_numpy(ht)


def off(x, ref):
    x = x.double().cpu()
    return float((x - ref).norm() / ref.norm())


@pytest.mark.parametrize("T", [1, 5, 150])
def test_layer_against_the_plain_form(T):
    layer = example.Int8DeltaLayer(256, 2, 4, 64, 64, seed=T)
    gen = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(2, T, 256, device="cuda", generator=gen).bfloat16()
    stream = torch.randn(2, T, 256, device="cuda", generator=gen).bfloat16()
    state = 0.3 * torch.randn(2, 4, 64, 64, device="cuda", generator=gen)
    want, s, ht = plain(layer, x, stream, state)
    note(f"int8 layer T={T}")
    y = layer(x, stream, state)
    torch.cuda.synchronize()
    assert torch.equal(stream, s)
    assert off(state, ht) < 5e-3
    assert off(y, want) < 0.044


def test_prompt_then_tokens():
    """A prompt and then single tokens give what one longer prompt gives."""
    layer = example.Int8DeltaLayer(256, 2, 4, 64, 64, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(1, 40, 256, device="cuda", generator=gen).bfloat16()
    stream = torch.randn(1, 40, 256, device="cuda", generator=gen).bfloat16()
    one, two = layer.zero_state(1), layer.zero_state(1)
    note("int8 layer, prompt then tokens")
    whole = layer(x, stream.clone(), one)
    parts = [layer(x[:, :32].contiguous(), stream[:, :32].contiguous(), two)]
    parts += [layer(x[:, t:t + 1].contiguous(), stream[:, t:t + 1].contiguous(), two) for t in range(32, 40)]
    torch.cuda.synchronize()
    assert off(torch.cat(parts, 1), whole.double().cpu()) < 0.044
    assert off(two, one.double().cpu()) < 5e-3

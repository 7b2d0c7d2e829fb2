"""A gated delta rule layer with 8-bit projections, as a server runs it: a prompt in one call, then
one token at a time, the recurrent state carried in place.

    python examples/int8_layer.py            # needs an MI355X and the built library

Per call: add_rmsnorm_i8 (residual stream, int8 activations), two matmul_i8 (q, k, v and the
output gate in bf16; decay and beta logits in fp32), the delta rule (chunked prefill, or the
decode step for one token), gated_rmsnorm_i8 and the output projection, another matmul_i8.
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_70_amd as gdr  # noqa: E402


class Int8DeltaLayer:
    """Random weights of the layer's shapes, int8 with a scale for each output channel."""

    def __init__(self, hidden, HK, HV, dk, dv, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        self.hidden, self.HK, self.HV, self.dk, self.dv = hidden, HK, HV, dk, dv

        def weights(rows, cols, gain=1.0):
            return gdr.quantize_rows_i8(gain * cols ** -0.5 * torch.randn(rows, cols, device=device, generator=gen))

        self.norm = torch.ones(hidden, device=device, dtype=torch.bfloat16)
        self.head_norm = torch.ones(dv, device=device)
        self.w_in, self.w_in_scale = weights(2 * HK * dk + 2 * HV * dv, hidden)
        self.w_in_scale[: HK * dk] *= dk ** -0.5  # the query's scale, in its channels' scales
        self.w_gate, self.w_gate_scale = weights(HV * dk + HV, hidden)
        self.gate_bias = torch.zeros(HV * dk + HV, device=device)
        self.gate_bias[: HV * dk] = -3.0          # slow decays
        self.w_out, self.w_out_scale = weights(hidden, HV * dv)

    def zero_state(self, B):
        return torch.zeros(B, self.HV, self.dk, self.dv, device=self.norm.device)

    def __call__(self, x, stream, state):
        """x: this layer's input to add to the residual ``stream``, both ``[B, T, hidden]`` bf16.
        Updates ``stream`` and ``state`` in place and returns the layer's output."""
        B, T, _ = x.shape
        HK, HV, dk, dv = self.HK, self.HV, self.dk, self.dv
        q8, s8, _ = gdr.add_rmsnorm_i8(x, self.norm, residual=stream, out_residual=stream)
        q, k, v, z = gdr.matmul_i8(q8, s8, self.w_in, self.w_in_scale, out=(HK * dk, HK * dk, HV * dv, HV * dv))
        a, b = gdr.matmul_i8(q8, s8, self.w_gate, self.w_gate_scale, bias=self.gate_bias, out=(HV * dk, HV),
                             out_dtype=torch.float32)
        args = (q.view(B, T, HK, dk), k.view(B, T, HK, dk), v.view(B, T, HV, dv), a.view(B, T, HV, dk), b.sigmoid_())
        if T == 1:
            o = gdr.decode_step(*args, state, k_l2norm=True, g_softplus=True)
        else:
            o, _ = gdr.forward(*args, h0=state, ht=state, k_l2norm=True, g_softplus=True)
        q8, s8 = gdr.gated_rmsnorm_i8(o, z.view(B, T, HV, dv), self.head_norm)
        return gdr.matmul_i8(q8, s8, self.w_out, self.w_out_scale)


def main():
    B, T, steps = 1, 4097, 64
    layer = Int8DeltaLayer(4096, 16, 32, 128, 128)
    x = torch.randn(B, T, 4096, device="cuda", dtype=torch.bfloat16)
    stream = torch.randn_like(x)
    for name, tokens, reps in (("prompt", T, 10), ("token", 1, steps)):
        xs, ss = x[:, :tokens].contiguous(), stream[:, :tokens].contiguous()
        state = layer.zero_state(B)
        for _ in range(3):
            y = layer(xs, ss, state)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            y = layer(xs, ss, state)
        torch.cuda.synchronize()
        t = (time.perf_counter() - t) / reps
        print(f"{name}: {tokens} token(s), {t * 1e6:.1f} us a layer, output {tuple(y.shape)} "
              f"rms {y.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()

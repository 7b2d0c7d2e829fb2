"""How calls of the 8-bit operators go: the memory of new outputs, streams given by handle, errors."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gpu_util import note

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def inputs(M, D, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    x, r = (torch.randn(M, D, device="cuda", generator=gen).to(BF) for _ in range(2))
    w, ws = gdr.quantize_rows_i8(torch.randn(64, D, device="cuda", generator=gen))
    return x, r, torch.ones(D, dtype=BF, device="cuda"), w, ws


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_new_outputs_on_another_stream(given):
    """Memory that was just freed on the current stream, where its last use may not have ended, does
    not become the output of a call on another one."""
    M, D = 4099, 1024
    x, r, nw, w, ws = inputs(M, D)
    want = gdr.add_rmsnorm_i8(x, nw, residual=r)
    y_want = gdr.matmul_i8(want[0], want[1], w, ws, out=(24, 40), out_dtype=F32)
    side = torch.cuda.Stream()
    s = side if given == "stream" else side.cuda_stream
    note(f"outputs on another stream, {given}")
    freed = [torch.empty_like(t) for t in (*want, *y_want)]
    places = {t.data_ptr() for t in freed}
    del freed
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.add_rmsnorm_i8(x, nw, residual=r, stream=s)
    y = gdr.matmul_i8(got[0], got[1], w, ws, out=(24, 40), out_dtype=F32, stream=s)
    assert not places & {t.data_ptr() for t in (*got, *y)}
    side.synchronize()
    for a, b in zip((*got, *y), (*want, *y_want)):
        assert torch.equal(a, b)


def test_default_stream_by_handle():
    """Handle 0, given while another stream is the current one: the default stream, whose memory new
    outputs are then of."""
    M, D = 4099, 1024
    x, r, nw, w, ws = inputs(M, D)
    want = gdr.add_rmsnorm_i8(x, nw, residual=r)
    note("default stream by its handle")
    freed = [torch.empty_like(t) for t in want]
    places = {t.data_ptr() for t in freed}
    del freed
    with torch.cuda.stream(torch.cuda.Stream()):
        got = gdr.add_rmsnorm_i8(x, nw, residual=r, stream=0)
    torch.cuda.synchronize()
    assert places & {t.data_ptr() for t in got}
    for a, b in zip(got, want):
        assert torch.equal(a, b)

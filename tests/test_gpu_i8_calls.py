"""How calls of the 8-bit operators go: the memory of new outputs, streams given by handle, errors."""
import ctypes

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


class FailingLibrary:
    """Entry points that fail as where HIP reports an error, and count the calls of each."""

    def __init__(self):
        self.calls = []
        self.kept = {}
        for name, n in (("gdr_add_rmsnorm_i8", 8), ("gdr_gated_rmsnorm_i8", 7), ("gdr_matmul_i8", 8)):
            self.kept[name] = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * n)(self.entry(name))
            setattr(self, name, self.entry(name))

    def entry(self, name):
        def failing(*args):
            self.calls.append(name)
            return 7
        return failing

    def addresses(self):
        return [ctypes.cast(self.kept[n], ctypes.c_void_p).value
                for n in ("gdr_add_rmsnorm_i8", "gdr_gated_rmsnorm_i8", "gdr_matmul_i8")]

    gdr_status_str = staticmethod(lambda status: b"a HIP call failed")


def test_a_failed_launch_is_not_tried_again(monkeypatch):
    """Part of a call may have run when a launch fails: adding a residual in place again would add it
    twice.  (The library is replaced by one that launches nothing.)"""
    qz = gdr.quantized
    M, D = 3, 64
    x, r, nw, w, ws = inputs(M, D)
    q, s, h = torch.empty(M, D, device="cuda", dtype=I8), torch.empty(M, device="cuda"), torch.empty_like(x)
    y = torch.empty(M, 64, device="cuda")
    o = torch.empty(M, 2, 32, device="cuda")
    qz._binding()
    L, bad = qz._lib(), FailingLibrary()
    real = [ctypes.cast(f, ctypes.c_void_p).value for f in (L.gdr_add_rmsnorm_i8, L.gdr_gated_rmsnorm_i8, L.gdr_matmul_i8)]
    calls = {"gdr_add_rmsnorm_i8": lambda: gdr.add_rmsnorm_i8(x, nw, residual=r, q=q, scale=s, out_residual=r),
             "gdr_gated_rmsnorm_i8": lambda: gdr.gated_rmsnorm_i8(o, o, torch.ones(32, device="cuda"), q=q, scale=s),
             "gdr_matmul_i8": lambda: gdr.matmul_i8(q, s, w, ws, out=y)}
    try:
        qz._B.bind(*bad.addresses(), qz._current_device, qz._raw_stream)
        monkeypatch.setattr(qz, "_L", bad)
        for name, call in calls.items():
            bad.calls.clear()
            with pytest.raises(gdr.GdrError) as e:
                call()
            assert e.value.status == 7 and bad.calls == [name]
    finally:
        qz._B.bind(*real, qz._current_device, qz._raw_stream)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [96, 333, 4096])
def test_streams_side_by_side(D, dtype):
    """Input, residual and new residual stream as column ranges of one array, which is written nowhere
    else."""
    M = 7
    gen = torch.Generator("cuda").manual_seed(D)
    wide = torch.randn(M, 3 * D + 2, device="cuda", generator=gen).to(dtype)
    w = torch.rand(D, device="cuda", generator=gen).to(dtype)
    before = wide.clone()
    x, out, r = wide[:, :D], wide[:, D:2 * D], wide[:, 2 * D:3 * D]
    want = gdr.add_rmsnorm_i8(x.contiguous(), w, residual=r.contiguous())
    note(f"streams side by side D={D} {dtype}")
    got = gdr.add_rmsnorm_i8(x, w, residual=r, out_residual=out)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    before[:, D:2 * D] = want[2]
    assert torch.equal(wide, before)


def test_capture_on_a_forked_stream():
    """Calls given a stream that joined a capture, with new outputs: replays follow their inputs."""
    M, D = 70, 512
    x, r, nw, w, ws = inputs(M, D)
    gdr.add_rmsnorm_i8(x, nw, residual=r)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    note("capture on a forked stream")
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        q, s, h = gdr.add_rmsnorm_i8(x, nw, residual=r, stream=side)
        y, z = gdr.matmul_i8(q, s, w, ws, out=(24, 40), out_dtype=F32, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for i in range(3):
        x.copy_(inputs(M, D, seed=10 + i)[0])
        g.replay()
        torch.cuda.synchronize()
        want = gdr.add_rmsnorm_i8(x, nw, residual=r)
        y_want = gdr.matmul_i8(want[0], want[1], w, ws, out=(24, 40), out_dtype=F32)
        for a, b in zip((q, s, h, y, z), (*want, *y_want)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()

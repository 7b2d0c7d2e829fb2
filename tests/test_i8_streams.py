"""Streams and memory of the 8-bit operators' binding, on the host: tensors that say they are on a
GPU, an allocator that notes from which stream's memory a tensor is taken and which streams it is
kept for, and a library that does nothing."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gated_delta_rule_70_amd import quantized as qz

HERE, THERE = 111, 222   # handles of the current stream and of another one
NEW = 333                # and of one that nobody uses


class Gpu(torch.Tensor):
    is_cuda = True
    taken_from, kept_for = None, ()

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.kept_for = (*self.kept_for, s.cuda_stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class NoLibrary:
    gdr_add_rmsnorm_i8 = gdr_gated_rmsnorm_i8 = gdr_matmul_i8 = staticmethod(lambda *a: 0)


@pytest.fixture
def machine(monkeypatch):
    active, empty = [HERE], torch.empty

    def set_stream(s):
        active[0] = s.cuda_stream

    def take(*a, **kw):
        t = empty(*a, **kw).as_subclass(Gpu)
        t.taken_from = active[0]
        return t

    monkeypatch.setattr(torch, "empty", take)
    monkeypatch.setattr(torch.cuda, "set_stream", set_stream)
    # torch's, given the handle 0, is a new stream
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle or NEW))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(active[0]))
    monkeypatch.setattr(qz, "_current_device", lambda: 0)
    monkeypatch.setattr(qz, "_raw_stream", lambda dev: active[0])
    monkeypatch.setattr(qz, "_L", NoLibrary)
    monkeypatch.setattr(qz, "_B", qz._NoBinding)


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Gpu)


def i8(*shape):
    return gpu(*shape, dtype=torch.int8)


CALLS = {
    "norm": lambda s: gdr.add_rmsnorm_i8(gpu(3, 64), gpu(64), residual=gpu(3, 64), stream=s),
    "gated": lambda s: gdr.gated_rmsnorm_i8(gpu(3, 2, 32), gpu(3, 2, 32), gpu(32), stream=s),
    "product": lambda s: [gdr.matmul_i8(i8(3, 64), gpu(3), i8(20, 64), gpu(20), stream=s)],
    "outputs": lambda s: gdr.matmul_i8(i8(3, 64), gpu(3), i8(20, 64), gpu(20), out=(8, 12), stream=s),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [THERE, Stream(THERE)], ids=["handle", "stream"])
def test_new_outputs_on_another_stream(call, stream, machine):
    """They come from the memory of the stream that writes them (the current one's may still be in
    use by work that this stream does not wait for), and are kept for the current one too."""
    for t in CALLS[call](stream):
        assert t.taken_from == THERE and HERE in t.kept_for


@pytest.mark.parametrize("given", [False, True], ids=["new", "given"])
def test_inputs_are_kept_for_the_stream(given, machine):
    a, sa, w, sw, b = i8(3, 64), gpu(3), i8(20, 64), gpu(20), gpu(20)
    outs = [gpu(3, 8), gpu(3, 12)] if given else (8, 12)
    gdr.matmul_i8(a, sa, w, sw, bias=b, out=outs, stream=THERE)
    assert all(THERE in t.kept_for for t in (a, sa, w, sw, b, *(outs if given else ())))


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [HERE, Stream(HERE)], ids=["handle", "stream"])
def test_new_outputs_on_the_current_stream(call, stream, machine):
    for t in CALLS[call](stream):
        assert t.taken_from == HERE and t.kept_for == ()


def test_given_tensors_on_another_stream(machine):
    x, w, r, q, s, o = gpu(3, 64), gpu(64), gpu(3, 64), i8(3, 64), gpu(3), gpu(3, 64)
    gdr.add_rmsnorm_i8(x, w, residual=r, q=q, scale=s, out_residual=o, stream=THERE)
    assert all(t.kept_for == (THERE,) for t in (x, w, r, q, s, o))


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_stays(call, machine):
    CALLS[call](THERE)
    assert torch.cuda.current_stream().cuda_stream == HERE


def test_the_current_stream_stays_after_a_refusal(machine):
    with pytest.raises(ValueError, match="weight must be"):
        gdr.add_rmsnorm_i8(gpu(3, 64), gpu(65), stream=THERE)
    assert torch.cuda.current_stream().cuda_stream == HERE


def test_handle_of_the_default_stream(machine):
    x, w = gpu(3, 64), gpu(64)
    q, s, _ = gdr.add_rmsnorm_i8(x, w, stream=0)
    assert x.kept_for == w.kept_for == (0,)
    assert q.taken_from == s.taken_from == 0

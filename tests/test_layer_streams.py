"""Streams and memory of the layer operators' binding, on the host: tensors that say they are on a GPU, an
allocator that notes from which stream's memory a tensor is taken and which streams it is kept for, and a
library that does nothing (and wants a workspace for every scan)."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gated_delta_rule_70_amd import quantized as qz
from test_i8_streams import HERE, THERE, Stream, gpu, machine  # noqa: F401

BF = torch.bfloat16


class NoLibrary:
    gdr_causal_conv = gdr_qk_norm_rope = gdr_selective_scan_step = staticmethod(lambda *a: 0)
    gdr_selective_scan_workspace_bytes = staticmethod(lambda *a: 64)
    workspace = None

    @classmethod
    def gdr_selective_scan(cls, *a):
        cls.workspace = a[13]
        return 0


@pytest.fixture
def layer_machine(machine, monkeypatch):  # noqa: F811
    monkeypatch.setattr(qz, "_L", NoLibrary)
    made = []
    empty = torch.empty

    def noted(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    monkeypatch.setattr(torch, "empty", noted)
    return made


def b(*shape):
    return gpu(*shape, dtype=BF)


CALLS = {
    "conv": lambda s: gdr.causal_conv(b(2, 5, 64), b(64, 4), state=b(2, 3, 64), stream=s),
    "conv_outs": lambda s: gdr.causal_conv(b(2, 5, 64), b(64, 4), out=(24, 40), stream=s),
    "conv_step": lambda s: gdr.causal_conv_step(b(2, 64), b(64, 4), b(2, 3, 64), out=[24, 40], stream=s),
    "qk": lambda s: gdr.qk_norm_rope(b(5, 4, 64), b(5, 2, 64), stream=s),
    "scan": lambda s: gdr.selective_scan(b(2, 5, 64), b(2, 5, 64), gpu(64, 16), b(2, 5, 16), b(2, 5, 16), stream=s),
    "scan_step": lambda s: gdr.selective_scan_step(b(2, 64), b(2, 64), gpu(64, 16), b(2, 16), b(2, 16), gpu(2, 64, 16), stream=s),
}


def flat(t):
    return [u for v in t for u in flat(v)] if isinstance(t, (tuple, list)) else [t]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [THERE, Stream(THERE)], ids=["handle", "stream"])
def test_new_outputs_on_another_stream(call, stream, layer_machine):
    """They come from the memory of the stream that writes them and are kept for the current one too."""
    for t in flat(CALLS[call](stream)):
        assert t.taken_from == THERE and HERE in t.kept_for
    assert torch.cuda.current_stream().cuda_stream == HERE


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [None, HERE])
def test_new_outputs_on_the_current_stream(call, stream, layer_machine):
    for t in flat(CALLS[call](stream)):
        assert t.taken_from == HERE


@pytest.mark.parametrize("given", [False, True])
def test_workspace_on_another_stream(given, layer_machine):
    """Also where every output is given; the library gets it, and it is kept for the stream that writes it."""
    x, h = b(2, 5, 64), gpu(2, 64, 16)
    outs = dict(out=b(2, 5, 64), ht=h) if given else {}
    gdr.selective_scan(x, b(2, 5, 64), gpu(64, 16), b(2, 5, 16), b(2, 5, 16), stream=THERE, **outs)
    work = [t for t in layer_machine if t.dtype is torch.uint8]
    assert len(work) == 1 and work[0].taken_from == THERE and work[0].data_ptr() == NoLibrary.workspace
    for t in outs.values():
        assert THERE in t.kept_for


def test_workspace_refusals(layer_machine):
    args = (b(2, 5, 64), b(2, 5, 64), gpu(64, 16), b(2, 5, 16), b(2, 5, 16))
    with pytest.raises(TypeError, match="workspace"):
        gdr.selective_scan(*args, workspace=gpu(64))
    with pytest.raises(ValueError, match="workspace"):
        gdr.selective_scan(*args, workspace=gpu(64, 2, dtype=torch.uint8)[:, 0])

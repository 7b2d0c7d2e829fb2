"""Outputs of the convolution given as any iterable, with a stream and without (on the host, as test_layer_streams.py)."""
import pytest

import gated_delta_rule_70_amd as gdr
from test_i8_streams import HERE, THERE, Stream, machine  # noqa: F401
from test_layer_streams import b, layer_machine  # noqa: F401

CALLS = {
    "prompt": (lambda out, s: gdr.causal_conv(b(2, 5, 64), b(64, 4), out=out, out_state=b(2, 3, 64), stream=s)[0], (2, 5)),
    "prompt_new_state": (lambda out, s: gdr.causal_conv(b(2, 5, 64), b(64, 4), out=out, stream=s)[0], (2, 5)),
    "single_tokens": (lambda out, s: gdr.causal_conv_step(b(2, 64), b(64, 4), b(2, 3, 64), out=out, stream=s), (2,)),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [None, HERE, THERE, Stream(THERE)], ids=["none", "current", "handle", "stream"])
@pytest.mark.parametrize("kind", [tuple, list, iter, lambda t: (u for u in t)], ids=["tuple", "list", "iterator", "generator"])
def test_given_outputs(call, stream, kind, layer_machine):  # noqa: F811
    run, lead = CALLS[call]
    outs = [b(*lead, 24), b(*lead, 40)]
    got = run(kind(outs), stream)
    assert isinstance(got, tuple) and [id(t) for t in got] == [id(t) for t in outs]
    if stream not in (None, HERE):  # memory of the current stream's is kept for the one that writes it
        assert all(THERE in t.kept_for for t in outs)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [None, THERE])
def test_counts_from_an_iterator(call, stream, layer_machine):  # noqa: F811
    run, lead = CALLS[call]
    got = run(iter((24, 40)), stream)
    assert [tuple(t.shape) for t in got] == [(*lead, 24), (*lead, 40)]
    assert all(t.taken_from == (stream or HERE) for t in got)

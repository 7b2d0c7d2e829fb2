"""Outputs of the 8-bit product given as any iterable, on another stream (on the host, as test_i8_streams.py)."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from test_i8_streams import THERE, gpu, machine  # noqa: F401


@pytest.mark.parametrize("kind", [tuple, list, iter], ids=["tuple", "list", "iterator"])
def test_given_outputs_are_kept_for_the_stream(kind, machine):  # noqa: F811
    """Memory of the current stream's is kept for the one that writes it."""
    outs = [gpu(3, 24), gpu(3, 40)]
    a, w = gpu(3, 16, dtype=torch.int8), gpu(64, 16, dtype=torch.int8)
    got = gdr.matmul_i8(a, gpu(3), w, gpu(64), out=kind(outs), stream=THERE)
    assert [id(t) for t in got] == [id(t) for t in outs] and all(THERE in t.kept_for for t in outs)

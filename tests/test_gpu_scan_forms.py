"""The values of every form of the selective scan over many tiles, against 64 bits (sizes in scan_forms.py)."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
import layer_reference as ref
from gpu_util import note
from scan_forms import FORMS, lengths
from test_gpu_layer import SENTINEL, cu_of, scan_inputs, scan_reference

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("case", FORMS, ids=lambda c: f"{c[0]}x{c[1]}{'-cut' if c[2] else ''}-{'packed' if lengths(c)[1] else 'dense'}-N{c[5]}")
def test_many_tiles(case):
    note(f"selective_scan {case}")
    (lens, packed), D, N, G, xt = lengths(case), *case[4:7], TYPES[case[7]]
    lead = (sum(lens),) if packed else (len(lens), lens[0])
    a = scan_inputs(lead, len(lens), D, N, G, xt, torch.float32, True, True, True, True, True, seed=31)
    a["dt_bias"] -= 2  # states that last for many tiles
    rows = torch.full((lead[0] + 8, *lead[1:], D), SENTINEL, dtype=xt, device="cuda")
    want, bound, end, end_bound = scan_reference(a, lens if packed else None)
    y, ht = gdr.selective_scan(**a, cu_seqlens=cu_of(lens) if packed else None, out=rows[4:-4])
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)
    assert (rows[:4] == SENTINEL).all() and (rows[-4:] == SENTINEL).all()

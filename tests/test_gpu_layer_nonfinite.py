"""Infinite inputs, steps, products and states of the selective scan: infinities where the formula has them, at
state counts that do and do not fill the lanes of a channel, in every form."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
import layer_reference as ref
from gpu_util import note

pytestmark = pytest.mark.gpu
F32 = torch.float32
INF = float("inf")
LARGEST = torch.finfo(F32).max


def inputs(B, T, D, N, seed):
    """fp32, B and C positive, so that states of one sign give a sum that is infinite and no NaN."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    return dict(x=torch.randn(B, T, D, generator=g), dt=0.2 * rand(B, T, D), A=-(0.1 + 2 * rand(D, N)), B=0.5 + rand(B, T, 1, N),
                C=1 + rand(B, T, 1, N), D=0.5 + rand(D), z=0.5 + rand(B, T, D), h0=torch.randn(B, D, N, generator=g))


def infinite(a, t):
    """Into the first sequence: an infinite input at token t of channel 3, an infinite step in channel 5, and in
    channel 7 finite ones whose product passes fp32's range, in a state that hardly decays."""
    a["x"][0, t, 3] = INF
    a["dt"][0, t, 5], a["x"][0, t, 5] = INF, 1.
    a["dt"][0, t, 7], a["x"][0, t, 7] = 4., 3e38
    a["A"][7] = -1e-6
    return a


def expected(a):
    """The formula's values, what passes fp32's range as infinity."""
    want, bound, end, end_bound = ref.scan(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], None, False, a["h0"])
    want, end = (torch.where(t.abs() > LARGEST, INF * t.sign(), t) for t in (want, end))
    return want, bound, end, end_bound


def on_gpu(a):
    return {k: v.cuda() for k, v in a.items()}


STATES = [1, 2, 3, 4, 5, 8, 10, 12, 15, 16, 17, 20, 32, 33, 64, 100, 128]


@pytest.mark.parametrize("N", STATES)
def test_single_tokens(N):
    """Token by token, the state in place."""
    note(f"selective_scan_step with infinities, N={N}")
    T, t0 = 6, 2
    a = infinite(inputs(2, T, 40, N, 1), t0)
    want, bound, end, end_bound = expected(a)
    assert not want.isnan().any() and want[0, t0:, [3, 5, 7]].isinf().all()
    g = on_gpu(a)
    state = g.pop("h0")
    for t in range(T):
        one = {k: v[:, t].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in g.items()}
        ref.close(gdr.selective_scan_step(**one, state=state), want[:, t], bound[:, t])
    ref.close(state, end, end_bound)


@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("B,T,D", [(2, 40, 40), (16, 37, 1000), (2, 700, 24)], ids=["sixteen_lanes", "four_lanes", "segments"])
def test_prompts(B, T, D, N):
    """Whole, with sixteen and (up to 16 states) with four lanes for a channel, and in segments; a token's y and
    every later one."""
    note(f"selective_scan with infinities {B}x{T}x{D}, N={N}")
    assert (gdr.selective_scan_workspace_bytes(B, T, D, N) > 0) == (T == 700)
    for t in (0, T // 2, T - 1):
        a = inputs(B, T, D, N, 2)
        a["z"] += 1.  # what passes the range stays past it at the gate
        if T == 700:
            a["dt"] *= 0.2  # states that last for segments
        infinite(a, t)
        want, bound, end, end_bound = expected(a)
        assert not want.isnan().any() and want[0, t:, [3, 5, 7]].isinf().all()
        y, ht = gdr.selective_scan(**on_gpu(a))
        ref.close(y, want, bound)
        ref.close(ht, end, end_bound)


@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("T", [60, 700])
def test_infinite_states(T, N):
    """A first state of infinity stays, however much of a finite one a segment would leave."""
    note(f"selective_scan from infinite states, T={T}, N={N}")
    a = inputs(2, T, 24, N, 3)
    a["h0"][0, 4, N - 1], a["h0"][1, 9, 0], a["h0"][1, 10, N // 2] = INF, -INF, INF
    a["A"][9], a["A"][10] = -60., -30.
    want, bound, end, end_bound = expected(a)
    assert not want.isnan().any() and want[0, :, 4].isinf().all() and want[1, :, 9:11].isinf().all()
    y, ht = gdr.selective_scan(**on_gpu(a))
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)


def test_a_state_that_a_token_wipes_out():
    """A token's factor below fp32's normal range counts as zero, and makes NaN of an infinite state; in segments
    as at once, wherever in them it is."""
    note("infinite states and factors of zero")
    N, D = 20, 24
    for T, t in ((60, 0), (60, 59), (700, 0), (700, 63), (700, 64), (700, 300), (700, 699)):
        a = inputs(1, T, D, N, 4)
        a["h0"][0, 2, 5], a["h0"][0, 6, 7], a["A"][6, 7] = INF, INF, -1e-3
        a["dt"][0, t] = 300.  # a factor of e^-600 and less, e^-0.3 in channel 6
        a["A"][2, 5] = -2.
        a["x"][0, t] = 0.
        y, ht = gdr.selective_scan(**on_gpu(a))
        bad = torch.zeros(T, D, dtype=torch.bool)
        bad[t:, 2] = True
        assert torch.equal(y[0].isnan().cpu(), bad)
        assert ht[0, 2, 5].isnan() and ht[0, 6, 7] == INF and ht.isnan().sum() == 1
        assert (y[0, :, 6] == INF).all() and (y[0, :t, 2] == INF).all()


@pytest.mark.parametrize("rate", [INF, LARGEST, 2.5e38])
@pytest.mark.parametrize("B,T,D", [(2, 3, 40), (16, 37, 1000), (2, 64, 40)])
def test_rates_past_the_range(B, T, D, rate):
    """A of infinity, and of values whose product with log2(e) passes fp32's range: a state that is not zero is
    infinite behind the first token, and stays so, whatever lies behind a sequence's end in a tile."""
    note(f"selective_scan {B}x{T}x{D}, A {rate}")
    a = inputs(B, T, D, 16, 5)
    a["A"][3, 2] = rate
    a["dt"] += 0.01
    a["h0"][:, 3, 2] = 1.
    y, ht = gdr.selective_scan(**on_gpu(a))
    assert (y[:, :, 3] == INF).all() and (ht[:, 3, 2] == INF).all()
    assert not y.isnan().any() and not ht.isnan().any() and ht.isinf().sum() == B
    one = {k: v[:, 0].contiguous().cuda() if k in ("x", "dt", "B", "C", "z") else v.cuda() for k, v in a.items() if k != "h0"}
    state = a["h0"].cuda()
    assert (gdr.selective_scan_step(**one, state=state)[:, 3] == INF).all() and (state[:, 3, 2] == INF).all()


@pytest.mark.parametrize("N", [3, 16, 20])
@pytest.mark.parametrize("B,T,D", [(2, 40, 40), (16, 37, 1000), (2, 700, 24)], ids=["sixteen_lanes", "four_lanes", "segments"])
def test_without_a_skip(B, T, D, N):
    """Where D is not given, an infinite input reaches y by the states alone, with a gate and without."""
    note(f"selective_scan with infinities and without D {B}x{T}x{D}, N={N}")
    for gate in (True, False):
        a = inputs(B, T, D, N, 6)
        a["z"] += 1.
        if T == 700:
            a["dt"] *= 0.2
        infinite(a, T // 2)
        a["D"], a["z"] = None, a["z"] if gate else None
        want, bound, end, end_bound = expected(a)
        assert not want.isnan().any() and want[0, T // 2:, [3, 5, 7]].isinf().all()
        g = {k: None if v is None else v.cuda() for k, v in a.items()}
        y, ht = gdr.selective_scan(**g)
        ref.close(y, want, bound)
        ref.close(ht, end, end_bound)
        state = g.pop("h0")
        for t in range(T // 2 + 2 if T == 40 else 0):
            one = {k: v[:, t].contiguous() if v is not None and k in ("x", "dt", "B", "C", "z") else v for k, v in g.items()}
            ref.close(gdr.selective_scan_step(**one, state=state), want[:, t], bound[:, t])


@pytest.mark.parametrize("N", [5, 16, 30])
def test_infinite_states_of_a_packed_batch(N):
    """In segments of several sequences, steps through softplus: states that stay, one that a token wipes out, and
    an infinite input, in the sequences that they belong to."""
    note(f"packed selective_scan in segments with infinite states, N={N}")
    lens, D = [700, 0, 3, 650], 24
    starts = [0, 700, 700, 703]
    assert gdr.selective_scan_workspace_bytes(len(lens), sum(lens), D, N, packed=True) > 0
    a = inputs(1, sum(lens), D, N, 7)
    a["h0"] = inputs(4, 1, D, N, 8)["h0"]
    a = {k: v[0] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    a["dt"], a["x"], a["z"] = 4 * a["dt"] - 3, a["x"].bfloat16(), a["z"].bfloat16()
    a["B"], a["C"] = a["B"].bfloat16(), a["C"].bfloat16()
    a["h0"][0, 4, 1], a["h0"][3, 9, 0], a["h0"][3, 2, 2] = INF, -INF, INF
    a["A"][9], a["A"][4, 1], a["A"][2, 2] = -60., -0.5, -2.
    gone = starts[3] + 200
    a["dt"][gone, 2] = 300.
    a["x"][starts[3] + 100, 3] = INF
    cu = torch.tensor([*starts, sum(lens)], dtype=torch.int32, device="cuda")
    y, ht = gdr.selective_scan(**on_gpu(a), dt_softplus=True, cu_seqlens=cu)
    y, ht = y.float().cpu(), ht.cpu()
    nan, inf = torch.zeros(y.shape, dtype=torch.bool), torch.zeros(y.shape, dtype=torch.bool)
    nan[gone:, 2] = True
    inf[:700, 4] = inf[starts[3]:, 9] = inf[starts[3]:gone, 2] = inf[starts[3] + 100:, 3] = True
    assert torch.equal(y.isnan(), nan) and torch.equal(y.isinf(), inf)
    assert (y[starts[3]:, 9] < 0).all() and (y[:700, 4] > 0).all() and (y[starts[3] + 100:, 3] > 0).all()
    hn, hi = torch.zeros(ht.shape, dtype=torch.bool), torch.zeros(ht.shape, dtype=torch.bool)
    hn[3, 2, 2] = hi[0, 4, 1] = hi[3, 9, 0] = True
    hi[3, 3] = True
    assert torch.equal(ht.isnan(), hn) and torch.equal(ht.isinf(), hi)


@pytest.mark.parametrize("T,t", [(60, 30), (700, 10), (700, 63), (700, 500)])
def test_a_token_wipes_out_where_its_segment_would_not(T, t):
    """A token's factor of 2^-144 and nothing near that around it: the half of its segment's is in range."""
    note(f"infinite states and a factor of zero in a segment's halves, T={T}, t={t}")
    N, D = 16, 24
    a = inputs(1, T, D, N, 9)
    a["h0"][0, 2, 5], a["A"][2, 5] = INF, -2.
    a["dt"][0, t], a["x"][0, t] = 50., 0.
    y, ht = gdr.selective_scan(**on_gpu(a))
    bad = torch.zeros(T, D, dtype=torch.bool)
    bad[t:, 2] = True
    assert torch.equal(y[0].isnan().cpu(), bad) and (y[0, :t, 2] == INF).all()
    assert ht[0, 2, 5].isnan() and ht.isnan().sum() == 1

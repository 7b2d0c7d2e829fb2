"""The operators before and beside the recurrence against their definitions in 64 bits
(tests/layer_reference.py, which derives how far they may be off)."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
import layer_reference as ref
from gpu_util import note

pytestmark = pytest.mark.gpu
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
SENTINEL = 77.0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()


def cu_of(lens, first=0):
    return (torch.tensor([0, *lens]).cumsum(0) + first).to(I32).cuda()


def spread(t, pad=3):
    """The same values as the first columns of a wider array, its rows begun off any alignment."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), SENTINEL, dtype=t.dtype, device=t.device)
    view = wide[..., 1:1 + t.shape[-1]]
    view.copy_(t)
    return view


# ---- causal_conv ---------------------------------------------------------------------------------

CONV = [
    # B, T, D, W, x, weight, bias, state, act, out
    (1, 1, 64, 4, BF, BF, False, True, "silu", None),
    (3, 2, 40, 4, BF, F32, True, True, "silu", (8, 32)),
    (2, 3, 129, 4, BF, BF, True, False, None, (1, 2, 126)),
    (2, 4, 7, 4, F32, F32, True, True, "silu", None),
    (1, 17, 1, 2, BF, BF, False, True, "silu", None),
    (5, 16, 96, 3, BF, BF, True, True, "silu", None),
    (2, 33, 1001, 3, F32, F32, False, True, None, (333, 668)),
    (1, 100, 520, 2, BF, F32, True, False, "silu", (256, 200, 64)),
    (2, 131, 2048, 4, BF, BF, False, True, "silu", (512, 512, 1024)),
    (3, 67, 48, 4, F32, F32, True, True, "silu", (6,) * 8),
]


def conv_inputs(B, T, D, W, xt, wt, bias, state, seed=0):
    g = gen(seed)
    return (randn(g, B, T, D, dtype=xt), randn(g, D, W, dtype=wt, scale=W ** -0.5), randn(g, D, dtype=wt) if bias else None,
            randn(g, B, W - 1, D, dtype=xt) if state else None)


@pytest.mark.parametrize("B,T,D,W,xt,wt,bias,state,act,out", CONV)
def test_conv(B, T, D, W, xt, wt, bias, state, act, out):
    note(f"causal_conv {B}x{T}x{D} W={W} {xt} {wt} out={out}")
    x, w, b, s = conv_inputs(B, T, D, W, xt, wt, bias, state)
    y, end = gdr.causal_conv(x, w, bias=b, state=s, activation=act, out=out)
    if out is not None:
        assert [p.shape[-1] for p in y] == list(out) and all(p.is_contiguous() for p in y)
        y = torch.cat(y, -1)
    want, bound, last = ref.conv(x, w, b, s, act == "silu")
    ref.close(y, want, bound)
    assert end.dtype == xt and torch.equal(ref.wide(end), last)


@pytest.mark.parametrize("lens", [[5], [0, 1, 2, 3, 4, 0, 17, 100, 0], [64, 64, 64], [3] * 40, [1, 0, 0, 0, 130]])
@pytest.mark.parametrize("xt,D,W", [(BF, 72, 4), (F32, 37, 3), (BF, 1030, 2)])
def test_conv_packed(lens, xt, D, W):
    """Rows before the first sequence and behind the last one are left as they were."""
    note(f"packed causal_conv {lens} {xt} D={D} W={W}")
    front, back = 4, 9
    g = gen(1)
    T = sum(lens)
    x = randn(g, front + T + back, D, dtype=xt)
    w, b, s = randn(g, D, W, dtype=xt), randn(g, D, dtype=xt), randn(g, len(lens), W - 1, D, dtype=xt)
    out = torch.full_like(x, SENTINEL)
    y, end = gdr.causal_conv(x, w, bias=b, state=s, cu_seqlens=cu_of(lens, front), out=out)
    assert y is out
    want, bound, last = ref.conv(x[front:front + T], w, b, s, True, lens)
    ref.close(y[front:front + T], want, bound)
    assert torch.equal(ref.wide(end), last)
    assert (y[:front] == SENTINEL).all() and (y[front + T:] == SENTINEL).all()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("xt,W,out", [(BF, 4, (24,)), (F32, 3, (29, 8)), (BF, 2, (5, 32)), (BF, 4, (17, 9, 3))])
def test_conv_long(packed, xt, W, out):
    """Tiles of eight rows, outputs of whole groups of channels, with a rest, and of fewer than eight."""
    note(f"long causal_conv {xt} W={W} {out} packed={packed}")
    D, lens = sum(out), [11000, 3, 0, 8, 21999]
    x, w, b, s = conv_inputs(len(lens) if packed else 3, 1, D, W, xt, xt, True, True, seed=8)
    g = gen(9)
    if packed:
        x = randn(g, sum(lens), D, dtype=xt)
        y, end = gdr.causal_conv(x, w, bias=b, state=s, cu_seqlens=cu_of(lens), out=out)
    else:
        x = randn(g, 3, 11003, D, dtype=xt)
        y, end = gdr.causal_conv(x, w, bias=b, state=s, out=out)
    want, bound, last = ref.conv(x, w, b, s, True, lens if packed else None)
    ref.close(torch.cat(y, -1), want, bound)
    assert torch.equal(ref.wide(end), last)


def test_rows_far_apart():
    """Rows 2^30 values apart: the third begins past 2^31 values, 2^32 bytes."""
    note("rows far apart")
    far, T = 2 ** 30 + 8, 3

    def spaced(*tail):
        n = torch.Size(tail).numel()
        return torch.empty((T - 1) * far + n, dtype=BF, device="cuda").as_strided((T, *tail), (far, *[torch.Size(tail[i + 1:]).numel() for i in range(len(tail))]))

    x, w, b, s = conv_inputs(1, T, 72, 4, BF, BF, True, True, seed=10)
    a_x, a_out = spaced(72), spaced(72)
    a_x.copy_(x[0])
    y, end = gdr.causal_conv(a_x[None], w, bias=b, state=s, out=a_out[None])
    want, bound, last = ref.conv(x, w, b, s, True)
    ref.close(y, want, bound)
    assert torch.equal(ref.wide(end), last)
    a = scan_inputs((1, T), 1, 72, 16, 1, BF, BF, True, True, True, True, True, seed=11)
    a_x.copy_(a["x"][0])
    want, bound, end, end_bound = scan_reference(a)
    y, ht = gdr.selective_scan(**{**a, "x": a_x[None]}, out=a_out[None])
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)
    q, k, qw, kw, cos, sin, pos = qk_inputs((T,), 2, 2, 32, 32, BF, BF, I32, seed=12)
    a_q, a_oq = a_x.as_strided((T, 2, 32), (far, 32, 1)), a_out.as_strided((T, 2, 32), (far, 32, 1))
    a_q.copy_(q)
    got = gdr.qk_norm_rope(a_q, k, qw, kw, cos, sin, positions=pos, out_q=a_oq)
    check_qk(got, q, k, qw, kw, cos, sin, pos, 1e-6, False)
    rows = [t.clone() for t in gdr.qk_norm_rope(q[0], k[0], qw, kw, cos, sin, positions=pos[0])]  # one token, without a dimension of tokens
    assert torch.equal(rows[0], got[0][0]) and torch.equal(rows[1], got[1][0])


def test_conv_strided_and_in_place():
    """A column range of a wider projection in, column ranges of one array out, the state in place."""
    note("strided causal_conv")
    x, w, b, s = conv_inputs(2, 37, 136, 4, BF, BF, True, True, seed=2)
    want, bound, last = ref.conv(x, w, b, s, True)
    whole = torch.full((2, 37, 200), SENTINEL, dtype=BF, device="cuda")
    (y0, y1), end = gdr.causal_conv(spread(x), w, bias=b, state=s, out=[whole[..., 3:75], whole[..., 90:154]], out_state=s)
    assert end is s and torch.equal(ref.wide(s), last)
    ref.close(torch.cat([y0, y1], -1), want, bound)
    left = torch.ones(200, dtype=torch.bool)
    left[3:75] = left[90:154] = False
    assert (whole[..., left.cuda()] == SENTINEL).all()


@pytest.mark.parametrize("B,D,W,xt,out", [(1, 8192, 4, BF, (2048, 2048, 4096)), (33, 72, 4, BF, None), (7, 37, 3, F32, (5, 32)), (300, 64, 2, BF, None)])
def test_conv_step(B, D, W, xt, out):
    """A token at a time gives bitwise what the whole sequence gives, the state in place."""
    note(f"causal_conv_step {B}x{D} W={W}")
    T = 6
    x, w, b, s = conv_inputs(B, T, D, W, xt, xt, True, True, seed=3)
    want, bound, last = ref.conv(x, w, b, s, True)
    y_all, end = gdr.causal_conv(x, w, bias=b, state=s)
    ref.close(y_all, want, bound)
    state, kept = s.clone(), s.clone()
    other = torch.empty_like(s)
    for t in range(T):
        before = state.clone()
        y = gdr.causal_conv_step(x[:, t].contiguous(), w, state, bias=b, out=out)
        y2 = gdr.causal_conv_step(x[:, t], w, before, bias=b, out_state=other)
        y = torch.cat(y, -1) if out else y
        assert torch.equal(y, y_all[:, t]) and torch.equal(y2, y) and torch.equal(other, state)
    assert torch.equal(state, end) and torch.equal(s, kept)
    y = gdr.causal_conv_step(x[:, 0], w, None, bias=b)
    ref.close(y, *[t[:, 0] for t in ref.conv(x[:, :1], w, b, None, True)[:2]])


@pytest.mark.parametrize("cut", [0, 1, 2, 3, 5, 20, 40, 41])
def test_conv_in_pieces(cut):
    x, w, b, s = conv_inputs(2, 41, 72, 4, BF, BF, True, True, seed=4)
    whole, end = gdr.causal_conv(x, w, bias=b, state=s)
    y0, mid = gdr.causal_conv(x[:, :cut].contiguous(), w, bias=b, state=s)
    y1, end2 = gdr.causal_conv(x[:, cut:].contiguous(), w, bias=b, state=mid)
    assert torch.equal(torch.cat([y0, y1], 1), whole) and torch.equal(end2, end)


def test_conv_non_finite():
    """Infinity and NaN reach the W outputs whose windows hold them, and no others."""
    x, w, b, s = conv_inputs(2, 50, 40, 4, F32, F32, True, True, seed=5)
    w = w.abs() + 0.1
    x[0, 10, 3], x[1, 20, 5], x[0, 30, 7], s[1, 2, 9] = float("inf"), float("nan"), float("-inf"), float("nan")
    for act in ("silu", None):
        y, _ = gdr.causal_conv(x, w, bias=b, state=s, activation=act)
        want, bound, _ = ref.conv(x, w, b, s, act == "silu")
        want = torch.where(want.isinf() & (want < 0) & (act == "silu"), float("nan"), want)
        ref.close(y, want, bound.nan_to_num(0.0, 0.0))
    assert y.isnan().sum() == 4 + 3 and y.isinf().sum() == 8


def test_conv_empty():
    x, w, b, s = conv_inputs(3, 0, 24, 4, BF, BF, True, True, seed=6)
    y, end = gdr.causal_conv(x, w, bias=b, state=s)
    assert y.shape == (3, 0, 24) and torch.equal(end, s)
    y, end = gdr.causal_conv(x, w, bias=b)
    assert (end == 0).all()
    y, end = gdr.causal_conv(x[:0], w, bias=b, want_state=False)
    assert y.shape == (0, 0, 24) and end is None


def test_conv_boundaries_of_anything():
    """Whatever cu_seqlens holds, nothing outside the tensors is touched and other sequences keep their results."""
    note("causal_conv with boundaries out of range")
    D, W, T = 40, 4, 64
    g = gen(7)
    x, w, s = randn(g, T, D, dtype=BF), randn(g, D, W, dtype=BF), randn(g, 4, W - 1, D, dtype=BF)
    for cu in ([-5, 20, 10, 200, 300], [0, 0, 2 ** 31 - 1, -2 ** 31, 64], [70, 80, 90, 100, 110]):
        room = torch.full((3 * T, D), SENTINEL, dtype=BF, device="cuda")
        gdr.causal_conv(x, w, state=s, cu_seqlens=torch.tensor(cu, dtype=I32, device="cuda"), out=room[T:2 * T])
        assert (room[:T] == SENTINEL).all() and (room[2 * T:] == SENTINEL).all()


# ---- qk_norm_rope ----------------------------------------------------------------------------------

QK = [
    # lead, HQ, HK, d, rotated, dtype, weights, interleaved, positions
    ((1,), 16, 16, 128, 128, BF, BF, False, I32),
    ((33,), 32, 16, 128, 128, BF, F32, False, I32),
    ((3, 21), 4, 1, 64, 64, BF, BF, False, None),
    ((77,), 7, 3, 80, 80, F32, F32, False, I64),
    ((40,), 8, 8, 256, 64, BF, BF, False, I32),
    ((2, 9), 5, 2, 32, 32, BF, BF, True, I64),
    ((65,), 3, 3, 128, 96, F32, F32, True, I32),
    ((19,), 2, 1, 26, 10, BF, BF, False, I32),
    ((19,), 2, 1, 27, 2, F32, F32, True, None),
    ((50,), 4, 4, 96, 48, BF, None, False, I32),
    ((12,), 1, 1, 512, 512, BF, F32, False, I32),
    ((12,), 2, 2, 400, 272, BF, F32, True, I32),
    ((9,), 3, 2, 1, 0, BF, BF, False, None),
    ((7,), 3, 2, 512, 8, BF, BF, False, I32),
    ((7,), 2, 2, 501, 98, F32, F32, True, I32),
    ((7,), 2, 2, 500, 500, F32, F32, False, I32),
    ((7,), 5, 2, 90, 90, BF, BF, False, I32),
    ((7,), 5, 2, 90, 90, BF, F32, True, I32),
    ((70,), 9, 2, 65, 34, BF, BF, False, I64),
    ((70,), 20, 2, 33, 18, BF, BF, True, I64),
    ((70,), 20, 2, 17, 2, F32, F32, True, I64),
    ((70,), 20, 2, 128, 66, BF, BF, False, I64),
    ((301,), 16, 4, 128, 0, BF, BF, False, None),
    ((5,), 2, 2, 16, 16, BF, BF, False, I32),
    ((130,), 6, 2, 112, 32, F32, F32, False, I32),
    ((0,), 2, 2, 64, 64, BF, BF, False, None),
]


def qk_inputs(lead, HQ, HK, d, rotated, dtype, wt, positions, seed=0):
    g = gen(seed)
    q, k = (randn(g, *lead, H, d, dtype=dtype, scale=3.0) for H in (HQ, HK))
    qw, kw = (None, None) if wt is None else (1 + randn(g, d, scale=0.2), 1 + randn(g, d, scale=0.2))
    qw, kw = (None if w is None else w.to(wt) for w in (qw, kw))
    length = 1000
    cos, sin = gdr.rope_table(length, rotated, device="cuda") if rotated else (None, None)
    pos = None if positions is None or not rotated else torch.randint(0, length, lead, generator=g).to(positions).cuda()
    return q, k, qw, kw, cos, sin, pos


def check_qk(got, q, k, qw, kw, cos, sin, pos, eps, interleaved):
    lead, rows = q.shape[:-2], max(1, q.shape[:-2].numel())
    if pos is None and len(lead) > 1:
        pos = torch.arange(lead[-1]).expand(lead).reshape(-1)
    for y, x, w in ((got[0], q, qw), (got[1], k, kw)):
        assert y.shape == x.shape and y.dtype == x.dtype
        flat = x.reshape(-1, *x.shape[-2:])
        want, bound = ref.qk(flat, w, cos, sin, None if pos is None else pos.reshape(-1), eps, interleaved)
        ref.close(y.reshape(flat.shape), want, bound)


@pytest.mark.parametrize("lead,HQ,HK,d,rotated,dtype,wt,interleaved,positions", QK)
def test_qk(lead, HQ, HK, d, rotated, dtype, wt, interleaved, positions):
    note(f"qk_norm_rope {lead} {HQ}+{HK}x{d} rotated={rotated} {dtype} {wt} {interleaved} {positions}")
    q, k, qw, kw, cos, sin, pos = qk_inputs(lead, HQ, HK, d, rotated, dtype, wt, positions)
    got = gdr.qk_norm_rope(q, k, qw, kw, cos, sin, positions=pos, eps=1e-5, interleaved=interleaved)
    check_qk(got, q, k, qw, kw, cos, sin, pos, 1e-5, interleaved)


@pytest.mark.parametrize("d,rotated,interleaved", [(64, 64, False), (128, 64, False), (48, 20, False), (64, 64, True), (30, 6, True)])
def test_qk_in_place_and_strided(d, rotated, interleaved):
    """q and k as column ranges of one projection's output, replaced there; the columns around them stay."""
    note(f"qk_norm_rope in place d={d} rotated={rotated}")
    HQ, HK, rows = 3, 2, 29
    q, k, qw, kw, cos, sin, pos = qk_inputs((rows,), HQ, HK, d, rotated, BF, BF, I32, seed=1)
    both = torch.full((rows, 1 + (HQ + HK + 1) * d), SENTINEL, dtype=BF, device="cuda")
    vq, vk = both[:, 1:1 + HQ * d].unflatten(1, (HQ, d)), both[:, 1 + HQ * d:1 + (HQ + HK) * d].unflatten(1, (HK, d))
    vq.copy_(q)
    vk.copy_(k)
    new = gdr.qk_norm_rope(vq, vk, qw, kw, cos, sin, positions=pos, interleaved=interleaved)
    check_qk(new, q, k, qw, kw, cos, sin, pos, 1e-6, interleaved)
    got = gdr.qk_norm_rope(vq, vk, qw, kw, cos, sin, positions=pos, interleaved=interleaved, out_q=vq, out_k=vk)
    assert got[0] is vq and torch.equal(vq, new[0]) and torch.equal(vk, new[1])
    assert (both[:, 0] == SENTINEL).all() and (both[:, 1 + (HQ + HK) * d:] == SENTINEL).all()


@pytest.mark.parametrize("d,rotated", [(64, 64), (64, 32), (30, 10)])
def test_qk_positions_outside(d, rotated):
    """Their rotated values are NaN, the others as ever; rows with the same position are alike."""
    note(f"positions outside the tables d={d}")
    q, k, qw, kw, cos, sin, _ = qk_inputs((8,), 2, 1, d, rotated, BF, BF, None, seed=2)
    for t in (I32, I64):
        pos = torch.tensor([0, 999, 1000, -1, 5, 5, 2 ** 31 - 1, -2 ** 31], dtype=t).cuda()
        got = gdr.qk_norm_rope(q, k, qw, kw, cos, sin, positions=pos)
        check_qk(got, q, k, qw, kw, cos, sin, pos, 1e-6, False)
    pos = torch.tensor([0, 1, 2 ** 40, -2 ** 63, 2 ** 32, 2 ** 32 + 1, 3, 4]).cuda()
    check_qk(gdr.qk_norm_rope(q, k, qw, kw, cos, sin, positions=pos), q, k, qw, kw, cos, sin, pos, 1e-6, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 26])
def test_qk_magnitudes(dtype, d):
    """Heads of zeros, from the smallest to the largest values, and with NaN or infinity."""
    note(f"qk magnitudes {dtype} d={d}")
    q, k, qw, kw, cos, sin, pos = qk_inputs((9,), 2, 2, d, d, dtype, dtype, I32, seed=3)
    scales = torch.tensor([1.0, 2.0 ** -120, 2.0 ** 120, 0.0, 2.0 ** -60, 2.0 ** 60, 1.0, 1.0, 2.0 ** -124]).cuda()
    q, k = ((t.float() * scales[:, None, None]).to(dtype) for t in (q, k))
    q[6, 0, 3], q[7, 1, 5] = float("inf"), float("nan")
    for eps in (0.0, 1e-6):
        got = gdr.qk_norm_rope(q, k, qw, kw, cos, sin, positions=pos, eps=eps)
        qr = q.clone()
        qr[6, 0], qr[7, 1] = float("nan"), float("nan")
        check_qk(got, qr, k, qw, kw, cos, sin, pos, eps, False)


@pytest.mark.parametrize("rows,HQ,HK,d", [(11000, 3, 1, 512), (2100, 5, 3, 16)])
def test_qk_many_heads(rows, HQ, HK, d):
    """More workgroups than the GPU holds at once, the last waves of a row with fewer heads."""
    note(f"qk_norm_rope {rows}x{HQ}+{HK}x{d}")
    q, k, qw, kw, cos, sin, pos = qk_inputs((rows,), HQ, HK, d, 16, BF, F32, I32, seed=5)
    check_qk(gdr.qk_norm_rope(q, k, qw, kw, cos, sin, positions=pos), q, k, qw, kw, cos, sin, pos, 1e-6, False)


def test_qk_length_one():
    """Keys of length one, as the delta rule takes them."""
    q, k, _, _, _, _, _ = qk_inputs((31,), 4, 4, 64, 0, F32, None, None, seed=4)
    w = torch.full((64,), 64 ** -0.5, device="cuda")
    q1, k1 = gdr.qk_norm_rope(q, k, w, w, eps=0.0)
    for a, b in ((q1, q), (k1, k)):
        want = ref.wide(b) / (ref.wide(b) ** 2).sum(-1, keepdim=True).sqrt()
        ref.close(a, want, 6 * ref.U * want.abs())  # the factor's rounding and two products; 64 ** -0.5 is exact


# ---- selective_scan --------------------------------------------------------------------------------

SCAN = [
    # B, T, D, N, G, x, dt, skip, z, bias, softplus, h0
    (1, 1, 16, 16, 1, BF, BF, True, True, True, True, True),
    (2, 5, 64, 16, 1, BF, F32, True, True, True, True, False),
    (1, 64, 48, 16, 1, BF, BF, True, True, True, True, True),
    (1, 65, 96, 16, 2, BF, BF, True, False, True, True, True),
    (3, 33, 100, 10, 1, F32, F32, False, False, False, False, True),
    (2, 17, 7, 1, 7, F32, F32, True, True, True, True, True),
    (1, 130, 33, 3, 3, BF, F32, True, True, True, True, False),
    (2, 40, 64, 17, 1, BF, BF, True, True, False, True, True),
    (1, 31, 40, 32, 2, F32, F32, True, True, True, True, True),
    (1, 50, 24, 64, 1, BF, BF, True, True, True, True, True),
    (1, 16, 20, 128, 2, F32, F32, True, True, True, True, True),
    (2, 15, 12, 100, 1, BF, BF, False, True, True, False, True),
    (9, 70, 130, 8, 1, BF, BF, True, True, True, True, True),
    (40, 20, 512, 16, 1, BF, BF, True, True, True, True, True),
    (3, 100, 257, 4, 1, BF, BF, True, True, True, True, True),
]


def scan_inputs(lead, seqs, D, N, G, xt, dtt, skip, z, bias, softplus, h0, seed=0):
    g = gen(seed)
    a = dict(x=randn(g, *lead, D, dtype=xt), A=-(0.1 + 4 * torch.rand(D, N, generator=g)).cuda(), B=randn(g, *lead, G, N, dtype=xt),
             C=randn(g, *lead, G, N, dtype=xt))
    a["dt"] = randn(g, *lead, D, dtype=dtt) if softplus else (0.2 * torch.rand(*lead, D, generator=g)).to(dtt).cuda()
    a["D"] = randn(g, D) if skip else None
    a["z"] = randn(g, *lead, D, dtype=xt) if z else None
    a["dt_bias"] = (randn(g, D) - 3) if bias and softplus else (0.05 * torch.rand(D, generator=g)).cuda() if bias else None
    a["dt_softplus"] = softplus
    a["h0"] = randn(g, seqs, D, N) if h0 else None
    return a


def scan_reference(a, lens=None):
    return ref.scan(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["dt_bias"], a["dt_softplus"], a["h0"], lens)


@pytest.mark.parametrize("B,T,D,N,G,xt,dtt,skip,z,bias,softplus,h0", SCAN)
def test_scan(B, T, D, N, G, xt, dtt, skip, z, bias, softplus, h0):
    note(f"selective_scan {B}x{T}x{D} N={N} G={G} {xt} {dtt}")
    a = scan_inputs((B, T), B, D, N, G, xt, dtt, skip, z, bias, softplus, h0)
    y, ht = gdr.selective_scan(**a)
    want, bound, end, end_bound = scan_reference(a)
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)
    if G == 1:  # without the dimension of groups
        a["B"], a["C"] = a["B"][:, :, 0], a["C"][:, :, 0]
        y1, h1 = gdr.selective_scan(**a)
        assert torch.equal(y, y1) and torch.equal(ht, h1)


@pytest.mark.parametrize("lens", [[5], [0, 1, 2, 16, 0, 17, 64, 65, 0], [3] * 30, [1, 0, 0, 129]])
@pytest.mark.parametrize("xt,D,N,G", [(BF, 72, 16, 1), (F32, 30, 5, 3), (BF, 40, 40, 1)])
def test_scan_packed(lens, xt, D, N, G):
    note(f"packed selective_scan {lens} {xt} D={D} N={N} G={G}")
    front, back, T = 4, 9, sum(lens)
    a = scan_inputs((front + T + back,), len(lens), D, N, G, xt, xt, True, True, True, True, True, seed=1)
    out = torch.full_like(a["x"], SENTINEL)
    y, ht = gdr.selective_scan(**a, cu_seqlens=cu_of(lens, front), out=out)
    assert y is out
    cut = {k: v[front:front + T] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    want, bound, end, end_bound = scan_reference(cut, lens)
    ref.close(y[front:front + T], want, bound)
    ref.close(ht, end, end_bound)
    assert (y[:front] == SENTINEL).all() and (y[front + T:] == SENTINEL).all()


SEGMENTS = [
    # B, T, D, N, G, x
    (1, 1000, 40, 16, 1, BF),
    (1, 4099, 24, 5, 3, F32),
    (3, 513, 70, 40, 1, F32),
    (2, 700, 17, 128, 1, BF),
    (1, 576, 33, 64, 1, F32),
]


@pytest.mark.parametrize("B,T,D,N,G,xt", SEGMENTS)
def test_scan_in_segments(B, T, D, N, G, xt):
    """Long sequences of few channels, that are cut; the workspace is given, or made, and may hold anything."""
    note(f"selective_scan in segments {B}x{T}x{D} N={N} G={G} {xt}")
    need = gdr.selective_scan_workspace_bytes(B, T, D, N, groups=G)
    assert need > 0
    a = scan_inputs((B, T), B, D, N, G, xt, F32, True, True, True, True, True, seed=9)
    a["dt_bias"] -= 2  # states that last for segments
    want, bound, end, end_bound = scan_reference(a)
    y, ht = gdr.selective_scan(**a)
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)
    room = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    y2, ht2 = gdr.selective_scan(**a, workspace=room[32:need + 32], ht=a["h0"])
    assert torch.equal(y2, y) and torch.equal(ht2, ht) and (room[:32] == 255).all() and (room[need + 32:] == 255).all()
    a["h0"] = None
    want, bound, end, end_bound = scan_reference(a)
    y, ht = gdr.selective_scan(**a)
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)


@pytest.mark.parametrize("lens", [[0, 1500, 3, 64, 700, 0], [2400], [800, 801, 799], [1, 1, 2300]])
@pytest.mark.parametrize("xt,D,N,G", [(BF, 40, 16, 1), (F32, 24, 5, 3)])
def test_scan_packed_in_segments(lens, xt, D, N, G):
    note(f"packed selective_scan in segments {lens} {xt} D={D} N={N}")
    front, back, T = 3, 900, sum(lens)
    assert gdr.selective_scan_workspace_bytes(len(lens), front + T + back, D, N, groups=G, packed=True) > 0
    a = scan_inputs((front + T + back,), len(lens), D, N, G, xt, xt, True, True, True, True, True, seed=10)
    a["dt_bias"] -= 2
    out = torch.full_like(a["x"], SENTINEL)
    y, ht = gdr.selective_scan(**a, cu_seqlens=cu_of(lens, front), out=out)
    cut = {k: v[front:front + T] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    want, bound, end, end_bound = scan_reference(cut, lens)
    ref.close(y[front:front + T], want, bound)
    ref.close(ht, end, end_bound)
    assert (y[:front] == SENTINEL).all() and (y[front + T:] == SENTINEL).all()


@pytest.mark.parametrize("lens", [[700, 0, 65, 1029, 3, 640], [1, 1, 1600, 33, 33]])
def test_scan_packed_in_segments_in_place(lens):
    """The state replaced by the last segment of each sequence, which the others begin from."""
    note(f"packed selective_scan in segments, in place {lens}")
    D, N, T = 20, 16, sum(lens) + 4000
    assert gdr.selective_scan_workspace_bytes(len(lens), T, D, N, packed=True) > 0
    a = scan_inputs((T,), len(lens), D, N, 1, BF, F32, True, True, True, True, True, seed=12)
    a["dt_bias"] -= 2
    cu = cu_of(lens, 0)
    cut = {k: v[:sum(lens)] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    want, bound, end, end_bound = scan_reference(cut, lens)
    y, ht = gdr.selective_scan(**a, cu_seqlens=cu)
    ref.close(y[:sum(lens)], want, bound)
    ref.close(ht, end, end_bound)
    for _ in range(5):
        state = a["h0"].clone()
        y2, h2 = gdr.selective_scan(**{**a, "h0": state}, cu_seqlens=cu, ht=state)
        assert h2 is state and torch.equal(state, ht) and torch.equal(y2[:sum(lens)], y[:sum(lens)])


@pytest.mark.parametrize("A,on,h0", [(2., 640, 0.), (1.5, 64, 2. ** -100), (-3., 640, 2. ** 100)])
def test_scan_in_segments_past_the_range_of_a_factor(A, on, h0):
    """Factors of a whole segment past fp32's range, states within it: zeros, or a small one."""
    note(f"selective_scan in segments, A {A}")
    T, D, N = 640, 16, 4
    assert gdr.selective_scan_workspace_bytes(1, T, D, N) > 0
    a = dict(x=torch.zeros(1, T, D, device="cuda"), dt=torch.zeros(1, T, D, device="cuda"),
             A=torch.full((D, N), A, device="cuda"), B=torch.ones(1, T, 1, N, device="cuda"), C=torch.ones(1, T, 1, N, device="cuda"),
             D=None, z=None, dt_bias=None, dt_softplus=False, h0=torch.full((1, D, N), h0, device="cuda"))
    a["dt"][:, :on] = 1.
    skip = 0
    if h0 == 0:  # nothing until the last 20 tokens, which stand for all
        skip = T - 20
        a["x"][:, skip:] = 1.
    want, bound, end, end_bound = scan_reference({k: v[:, skip:] if k in ("x", "dt", "B", "C") else v for k, v in a.items()})
    assert want.isfinite().all() and end.isfinite().all() and bound.isfinite().all()
    y, ht = gdr.selective_scan(**a)
    assert (y[:, :skip] == 0).all()
    ref.close(y[:, skip:], want, bound)
    ref.close(ht, end, end_bound)


@pytest.mark.parametrize("B,T,D,N,xt", [(17, 40, 1000, 16, BF), (64, 21, 520, 7, F32), (16, 35, 1024, 16, BF), (32, 21, 500, 13, F32)])
def test_scan_of_many_channels(B, T, D, N, xt):
    """Enough for four lanes a channel in some, sixteen in others."""
    note(f"selective_scan {B}x{T}x{D} N={N} {xt}")
    a = scan_inputs((B, T), B, D, N, 1, xt, xt, True, True, True, True, True, seed=11)
    want, bound, end, end_bound = scan_reference(a)
    y, ht = gdr.selective_scan(**a)
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)


def test_scan_packed_many_sequences():
    """Four lanes for a channel in a packed batch, sequences that end inside a tile."""
    note("packed selective_scan of 70 sequences")
    lens = [int(n) for n in torch.randint(0, 19, (70,), generator=gen(12))]
    D, T = 1000, sum(lens)
    a = scan_inputs((T + 5,), len(lens), D, 16, 1, BF, BF, True, True, True, True, True, seed=12)
    out = torch.full_like(a["x"], SENTINEL)
    y, ht = gdr.selective_scan(**a, cu_seqlens=cu_of(lens), out=out)
    cut = {k: v[:T] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    want, bound, end, end_bound = scan_reference(cut, lens)
    ref.close(y[:T], want, bound)
    ref.close(ht, end, end_bound)
    assert (y[T:] == SENTINEL).all()


@pytest.mark.parametrize("T,D", [(1, 40), (21, 40), (1100, 40), (21, 1024)])
def test_scan_without_memory(T, D):
    """A of -infinity: the state is the last token's input alone, whatever comes behind the sequence's end in
    a tile; in every form of the kernel."""
    B = 16 if D > 40 else 1
    a = scan_inputs((B, T), B, D, 16, 1, F32, F32, True, False, True, True, True, seed=13)
    a["A"][::2] = -float("inf")
    y, ht = gdr.selective_scan(**a)
    v = ref.wide(a["dt"]) + ref.wide(a["dt_bias"])
    step = torch.nn.functional.softplus(v)
    last = (step * ref.wide(a["x"]))[:, -1, ::2, None] * ref.wide(a["B"])[:, -1]
    # softplus (16 u), its argument's rounding (|v| u of a small value), two products
    bound = (18 + v.abs()[:, -1, ::2, None]) * ref.U * last.abs()
    assert not y.isnan().any() and not ht.isnan().any()
    ref.close(ht[:, ::2], last, bound)
    one = {k: v[:, -1] if k in ("x", "dt", "B", "C") else v for k, v in a.items() if k not in ("h0", "z")}
    end = torch.empty_like(ht)
    gdr.selective_scan_step(**one, state=a["h0"], out_state=end)
    ref.close(end[:, ::2], last, bound)


def test_packed_batch_of_nothing():
    a = scan_inputs((0,), 3, 24, 16, 1, BF, BF, True, True, True, True, True, seed=14)
    cu = torch.zeros(4, dtype=I32, device="cuda")
    y, ht = gdr.selective_scan(**a, cu_seqlens=cu)
    assert y.shape == (0, 24) and torch.equal(ht, a["h0"])
    x, w, b, s = conv_inputs(3, 0, 24, 4, BF, BF, True, True)
    y, end = gdr.causal_conv(x[0], w, bias=b, state=s, cu_seqlens=cu)
    assert y.shape == (0, 24) and torch.equal(end, s)


def test_scan_strided_and_in_place():
    """Inputs as column ranges of wider arrays, the output into one, the state in place."""
    note("strided selective_scan")
    a = scan_inputs((2, 37), 2, 72, 16, 2, BF, BF, True, True, True, True, True, seed=2)
    want, bound, end, end_bound = scan_reference(a)
    for k in ("x", "dt", "z"):
        a[k] = spread(a[k])
    bc = spread(torch.cat([a["B"].flatten(-2), a["C"].flatten(-2)], -1))
    a["B"], a["C"] = bc[..., :32].unflatten(-1, (2, 16)), bc[..., 32:].unflatten(-1, (2, 16))
    whole = torch.full((2, 37, 90), SENTINEL, dtype=BF, device="cuda")
    y, ht = gdr.selective_scan(**a, out=whole[..., 5:77], ht=a["h0"])
    assert ht is a["h0"]
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)
    assert (whole[..., :5] == SENTINEL).all() and (whole[..., 77:] == SENTINEL).all()


@pytest.mark.parametrize("B,D,N,G,xt,dtt", [(1, 4096, 16, 1, BF, BF), (33, 72, 16, 2, BF, F32), (5, 37, 10, 1, F32, F32),
                                            (70, 64, 64, 1, BF, BF), (3, 20, 128, 4, F32, F32), (2, 9, 1, 1, BF, BF), (17, 130, 7, 1, BF, BF),
                                            (8195, 5, 8, 1, BF, BF), (3, 70, 19, 1, BF, F32), (4, 33, 2, 1, F32, F32), (5, 20, 101, 1, BF, BF), (9, 30, 34, 2, F32, F32), (9, 40, 4, 1, F32, F32), (6, 30, 28, 2, BF, BF)])
def test_scan_step(B, D, N, G, xt, dtt):
    """Token by token within the whole sequence's bounds, the state in place."""
    note(f"selective_scan_step {B}x{D} N={N} G={G} {xt}")
    T = 4
    a = scan_inputs((B, T), B, D, N, G, xt, dtt, True, True, True, True, True, seed=3)
    want, bound, end, end_bound = scan_reference(a)
    state = a.pop("h0").clone()
    other = torch.empty_like(state)
    for t in range(T):
        one = {k: v[:, t] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
        before = state.clone()
        y = gdr.selective_scan_step(**one, state=state)
        ref.close(y, want[:, t], bound[:, t])
        y2 = gdr.selective_scan_step(**one, state=before, out_state=other)
        assert torch.equal(y, y2) and torch.equal(other, state)
    ref.close(state, end, end_bound)
    y = gdr.selective_scan_step(**one, state=None, out_state=other)
    first = {k: v[:, T - 1:] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    want, bound, end, end_bound = scan_reference({**first, "h0": None})
    ref.close(y, want[:, 0], bound[:, 0])
    ref.close(other, end, end_bound)


@pytest.mark.parametrize("cut", [0, 1, 16, 63, 64, 90])
def test_scan_in_pieces(cut):
    a = scan_inputs((2, 90), 2, 40, 16, 1, BF, BF, True, True, True, True, True, seed=4)
    want, bound, end, end_bound = scan_reference(a)
    parts = [{k: v[:, s].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()} for s in (slice(0, cut), slice(cut, 90))]
    y0, mid = gdr.selective_scan(**parts[0])
    y1, ht = gdr.selective_scan(**{**parts[1], "h0": mid})
    ref.close(torch.cat([y0, y1], 1), want, bound)
    ref.close(ht, end, end_bound)


@pytest.mark.parametrize("v", [-200.0, -90.0, -30.0, -8.0, 0.0, 8.0, 30.0, 90.0, 300.0])
def test_scan_steps_of_any_size(v):
    """softplus far from zero on either side, decays that leave nothing, and none at all."""
    a = scan_inputs((1, 20), 1, 32, 16, 1, F32, F32, True, True, False, True, True, seed=5)
    a["dt"] = a["dt"] * 0.1 + v
    a["A"][3], a["A"][4] = 0.0, -1e-30
    y, ht = gdr.selective_scan(**a)
    want, bound, end, end_bound = scan_reference(a)
    ref.close(y, want, bound)
    ref.close(ht, end, end_bound)


def test_scan_non_finite():
    """NaN and infinity stay in their channel and sequence, from their token on."""
    a = scan_inputs((2, 30), 2, 40, 16, 1, F32, F32, True, False, True, True, True, seed=6)
    a["x"][0, 10, 3], a["dt"][1, 20, 5], a["h0"][1, 7, 2] = float("nan"), float("nan"), float("nan")
    y, ht = gdr.selective_scan(**a)
    bad = torch.zeros(2, 30, 40, dtype=torch.bool)
    bad[0, 10:, 3] = bad[1, 20:, 5] = bad[1, :, 7] = True
    assert torch.equal(y.isnan().cpu(), bad) and not y.isinf().any()
    hb = torch.zeros(2, 40, 16, dtype=torch.bool)
    hb[0, 3] = hb[1, 5] = hb[1, 7, 2] = True
    assert torch.equal(ht.isnan().cpu(), hb)


def test_scan_empty():
    a = scan_inputs((3, 0), 3, 24, 16, 1, BF, BF, True, True, True, True, True, seed=7)
    y, ht = gdr.selective_scan(**a)
    assert y.shape == (3, 0, 24) and torch.equal(ht, a["h0"])
    y, ht = gdr.selective_scan(**{**a, "h0": None})
    assert (ht == 0).all()
    y, ht = gdr.selective_scan(**{k: v[:0] if k in ("x", "dt", "B", "C", "z", "h0") else v for k, v in a.items()}, want_state=False)
    assert y.shape == (0, 0, 24) and ht is None


def test_scan_boundaries_of_anything():
    note("selective_scan with boundaries out of range")
    T, D = 64, 40
    a = scan_inputs((T,), 4, D, 16, 1, BF, BF, True, True, True, True, True, seed=8)
    for cu in ([-5, 20, 10, 200, 300], [0, 0, 2 ** 31 - 1, -2 ** 31, 64], [70, 80, 90, 100, 110]):
        room = torch.full((3 * T, D), SENTINEL, dtype=BF, device="cuda")
        gdr.selective_scan(**a, cu_seqlens=torch.tensor(cu, dtype=I32, device="cuda"), out=room[T:2 * T])
        assert (room[:T] == SENTINEL).all() and (room[2 * T:] == SENTINEL).all()


@pytest.mark.parametrize("D", [40, 1200])
def test_entries_outside_the_batch(D):
    """Bounds of sequences that are none lead nowhere outside the tensors, in segments (few channels) or whole."""
    T, N, front = 1500, 16, 7
    for entries in ([-5, 900, 300, 10 ** 9], [T + 1, T + 2, T + 3, T + 4], [-3, -2, -1, 0], [1000, 500, 200, 2 ** 31 - 1]):
        note(f"packed operators, D {D}, bounds {entries}")
        cu = torch.tensor(entries, dtype=torch.int32, device="cuda")
        assert (gdr.selective_scan_workspace_bytes(3, T, D, N, packed=True) > 0) == (D == 40)
        a = scan_inputs((T,), 3, D, N, 1, BF, BF, True, True, True, True, True, seed=13)
        room = torch.full((front + T + front, D), SENTINEL, dtype=BF, device="cuda")
        ends = torch.full((5, D, N), SENTINEL, device="cuda")
        gdr.selective_scan(**a, cu_seqlens=cu, out=room[front:front + T], ht=ends[1:4])
        torch.cuda.synchronize()
        x, w, b, s = conv_inputs(3, 1, D, 4, BF, BF, True, True)
        room2, ends2 = torch.full_like(room, SENTINEL), torch.full((5, 3, D), SENTINEL, dtype=BF, device="cuda")
        gdr.causal_conv(a["x"], w, bias=b, state=s, cu_seqlens=cu, out=room2[front:front + T], out_state=ends2[1:4])
        torch.cuda.synchronize()
        for r in (room, room2):
            assert (r[:front] == SENTINEL).all() and (r[front + T:] == SENTINEL).all()
        for e in (ends, ends2):
            assert (e[0] == SENTINEL).all() and (e[4] == SENTINEL).all()

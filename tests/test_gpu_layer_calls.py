"""How calls of the operators before and beside the recurrence go (streams, graphs, the extension and the
Python path), and the operators run together as a layer runs them."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
import layer_reference as ref
from gated_delta_rule_70_amd import quantized as qz
from gpu_util import note

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed=0, B=2, T=70, D=136, N=16):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s, dtype=BF: torch.randn(*s, device="cuda", generator=g).to(dtype)
    cos, sin = gdr.rope_table(100, 32, device="cuda")
    a = dict(x=r(B, T, D), w=r(D, 4), cs=r(B, 3, D), dt=r(B, T, D), A=-torch.rand(D, N, device="cuda", generator=g) - 0.1,
             B=r(B, T, N), C=r(B, T, N), h=r(B, D, N, dtype=F32), q=r(B, T, 3, 64), k=r(B, T, 2, 64), cos=cos, sin=sin)
    long = dict(lx=r(1, 1100, 40), ldt=r(1, 1100, 40) - 4, lA=-torch.rand(40, N, device="cuda", generator=g), lB=r(1, 1100, N), lC=r(1, 1100, N))
    return a | long


def flat(t):
    return [u for v in t for u in flat(v)] if isinstance(t, (tuple, list)) else [t]


CALLS = {
    "conv": (lambda a, o, **k: gdr.causal_conv(a["x"], a["w"], state=a["cs"], out=o[:1], out_state=o[1], **k),
             lambda a, **k: gdr.causal_conv(a["x"], a["w"], state=a["cs"], **k)),
    "conv_step": (lambda a, o, **k: gdr.causal_conv_step(a["x"][0], a["w"], None, out=o[0], **k),
                  lambda a, **k: gdr.causal_conv_step(a["x"][0], a["w"], None, **k)),
    "qk": (lambda a, o, **k: gdr.qk_norm_rope(a["q"], a["k"], None, None, a["cos"], a["sin"], out_q=o[0], out_k=o[1], **k),
           lambda a, **k: gdr.qk_norm_rope(a["q"], a["k"], None, None, a["cos"], a["sin"], **k)),
    "scan": (lambda a, o, **k: gdr.selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], h0=a["h"], dt_softplus=True, out=o[0], ht=o[1], **k),
             lambda a, **k: gdr.selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], h0=a["h"], dt_softplus=True, **k)),
    "scan_in_segments": (lambda a, o, **k: gdr.selective_scan(a["lx"], a["ldt"], a["lA"], a["lB"], a["lC"], dt_softplus=True, out=o[0], ht=o[1], **k),
                         lambda a, **k: gdr.selective_scan(a["lx"], a["ldt"], a["lA"], a["lB"], a["lC"], dt_softplus=True, **k)),
    "scan_step": (lambda a, o, **k: gdr.selective_scan_step(a["x"][:, 5], a["dt"][:, 5], a["A"], a["B"][:, 5], a["C"][:, 5], a["h"], dt_softplus=True,
                                                            out=o[0], out_state=o[1], **k),
                  lambda a, **k: gdr.selective_scan_step(a["x"][:, 5], a["dt"][:, 5], a["A"], a["B"][:, 5], a["C"][:, 5], a["h"].clone(),
                                                         dt_softplus=True, **k)),
}


def outputs(name, a):
    """The results of a call that makes its own, and room for another's."""
    got = CALLS[name][1](a)
    want = flat(got)
    if name == "scan_step":
        want = [want[0], torch.empty_like(a["h"])]
        CALLS[name][0](a, want)
    return want, [torch.full_like(t, 7.0) for t in want]


@pytest.mark.parametrize("name", CALLS)
def test_python_path_and_extension(name, monkeypatch):
    """The extension takes the calls that it is for, and gives what the Python path gives."""
    note(f"{name}: extension and Python path")
    a = inputs()
    want, room = outputs(name, a)
    CALLS[name][0](a, room, stream=torch.cuda.current_stream())
    for t, w in zip(room, want):
        assert torch.equal(t, w)
    assert qz._binding() is not qz._NoBinding
    if name == "scan_in_segments":  # has no workspace to give
        CALLS[name][0](a, room, workspace=torch.empty(gdr.selective_scan_workspace_bytes(1, 1100, 40, 16), dtype=torch.uint8, device="cuda"))
        monkeypatch.setattr(gdr.layer, "_stream", None)
        room = [t.fill_(7.0) for t in room]
        CALLS[name][0](a, room, workspace=torch.empty(gdr.selective_scan_workspace_bytes(1, 1100, 40, 16), dtype=torch.uint8, device="cuda"))
    else:
        monkeypatch.setattr(gdr.layer, "_stream", None)  # what the Python path cannot do without
        room = [t.fill_(7.0) for t in room]
        CALLS[name][0](a, room)
    for t, w in zip(room, want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", ["stream", "handle", "current"])
def test_another_stream(name, given):
    """Work goes to the stream that is named, or to the current one; memory just freed on the current
    stream does not become an output of a call on another one."""
    note(f"{name} on another stream, {given}")
    a = inputs(1)
    want, room = outputs(name, a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    if given == "current":
        with torch.cuda.stream(side):
            CALLS[name][0](a, room)
            got = flat(CALLS[name][1](a))
    else:
        freed = [torch.empty_like(t) for t in want]
        places = {t.data_ptr() for t in freed}
        del freed
        s = side if given == "stream" else side.cuda_stream
        CALLS[name][0](a, room, stream=s)
        h = a["h"].clone()
        torch.cuda.synchronize()
        got = flat(CALLS[name][1](a | {"h": h}, stream=s))
        assert not places & {t.data_ptr() for t in got}
    side.synchronize()
    for t, w in zip(room, want):
        assert torch.equal(t, w)
    for t, w in zip(got, want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("name", CALLS)
def test_graph(name):
    """Captured and replayed with other inputs, with eager work and synchronizations between."""
    note(f"{name} captured")
    a = inputs(2)
    want, room = outputs(name, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        CALLS[name][0](a, room)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        CALLS[name][0](a, room)
    for i in range(4):
        b = inputs(3 + i)
        want, _ = outputs(name, b)
        for k in a:
            a[k].copy_(b[k])
        for t in room:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        for t, w in zip(room, want):
            assert torch.equal(t, w), i


def test_two_calls_at_once():
    """Scans in segments on two streams, each with memory of its own."""
    note("two scans in segments at once")
    a, b = inputs(8), inputs(9)
    wants = [flat(CALLS["scan_in_segments"][1](x)) for x in (a, b)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    gots = []
    for x, s in zip((a, b), sides):
        with torch.cuda.stream(s):
            gots.append([flat(CALLS["scan_in_segments"][1](x)) for _ in range(5)])
    torch.cuda.synchronize()
    for many, want in zip(gots, wants):
        for got in many:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tensors_of_another_device():
    a = inputs(10)
    with pytest.raises(ValueError, match="weight must be a GPU tensor"):
        gdr.causal_conv(a["x"], a["w"].cpu())
    with pytest.raises(ValueError, match="positions must be a GPU tensor"):
        gdr.qk_norm_rope(a["q"], a["k"], None, None, a["cos"], a["sin"], positions=torch.zeros(2, 70, dtype=torch.int32))
    with pytest.raises(ValueError, match="A must be a GPU tensor"):
        gdr.selective_scan(a["x"], a["dt"], a["A"].cpu(), a["B"], a["C"])


def test_overlapping_outputs():
    a = inputs(11)
    with pytest.raises(gdr.GdrError, match="overlap"):
        gdr.causal_conv(a["x"], a["w"], out=a["x"])
    with pytest.raises(gdr.GdrError, match="overlap"):
        gdr.selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], out=a["x"])
    with pytest.raises(gdr.GdrError, match="overlap"):
        gdr.qk_norm_rope(a["q"], a["q"], out_q=a["q"], out_k=torch.empty_like(a["q"]))


# ---- together --------------------------------------------------------------------------------------

HK, HV, DK, DV = 2, 4, 64, 64


def delta_layer(qkv, conv, state, pos, w, cos, sin, g, beta):
    """One layer's way from projection to recurrence, for a prompt or for single tokens."""
    B, T, _ = qkv.shape
    cols = (HK * DK, HK * DK, HV * DV)
    if T == 1:
        q, k, v = gdr.causal_conv_step(qkv[:, 0], w["conv"], conv, out=cols)
    else:
        (q, k, v), _ = gdr.causal_conv(qkv, w["conv"], state=conv, out=cols, out_state=conv)
    q, k, v = q.view(B, T, HK, DK), k.view(B, T, HK, DK), v.view(B, T, HV, DV)
    q, k = gdr.qk_norm_rope(q, k, w["q"], w["k"], cos, sin, positions=pos, eps=1e-6 / DK, out_q=q, out_k=k)
    if T == 1:
        return gdr.decode_step(q, k, v, g, beta, state)
    return gdr.chunk_prefill(q, k, v, g, beta, h0=state, ht=state)[0]


def test_delta_rule_layer():
    """Convolution, norm and rotation, delta rule: a prompt at once against the same tokens as a prompt and
    single tokens, and against 64 bits."""
    note("convolution, norm and rotation, delta rule")
    import oracle

    B, T, cut = 2, 80, 77
    g = torch.Generator("cuda").manual_seed(12)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    D = 2 * HK * DK + HV * DV
    qkv = r(B, T, D).to(BF)
    w = {"conv": (0.5 * r(D, 4)).to(BF), "q": torch.full((DK,), DK ** -1.0, device="cuda"), "k": torch.full((DK,), DK ** -0.5, device="cuda")}
    cos, sin = gdr.rope_table(T, 32, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
    gate, beta = -torch.nn.functional.softplus(r(B, T, HV, DK)), r(B, T, HV).sigmoid()
    runs = []
    for pieces in ([(0, T)], [(0, cut)] + [(t, t + 1) for t in range(cut, T)]):
        conv, state = torch.zeros(B, 3, D, device="cuda", dtype=BF), torch.zeros(B, HV, DK, DV, device="cuda")
        o = [delta_layer(qkv[:, a:b].contiguous(), conv, state, pos[:, a:b].contiguous(), w, cos, sin, gate[:, a:b].contiguous(),
                         beta[:, a:b].contiguous()) for a, b in pieces]
        runs.append((torch.cat(o, 1), state, conv))
    y, _, last = ref.conv(qkv, w["conv"], None, None, True)
    y = y.to(BF)
    q, k = (ref.qk(t.reshape(B * T, HK, DK), w[n], cos, sin, pos.reshape(-1), 1e-6 / DK, False)[0].to(BF)
            for n, t in (("q", y[..., :HK * DK]), ("k", y[..., HK * DK:2 * HK * DK])))
    o_ref, s_ref = oracle.sequential(q.view(B, T, HK, DK), k.view(B, T, HK, DK), y[..., 2 * HK * DK:].reshape(B, T, HV, DV).contiguous(),
                                     gate.cpu(), beta.cpu(), None)
    for o, state, conv in runs:
        assert torch.equal(ref.wide(conv), last)
        # the recurrence's own bar, and bf16 inputs that may round the other way here and there
        assert oracle.rel_err(o.double().cpu().numpy(), o_ref) < 2e-3 + 2.0 ** -8
        assert oracle.rel_err(state.double().cpu().numpy(), s_ref) < 2e-3 + 2.0 ** -8


def test_scan_layer():
    """Convolution and scan over a packed batch, then single tokens, against 64 bits."""
    note("convolution, scan")
    lens, steps, D, N = [33, 0, 80], 3, 72, 16
    S, T = len(lens), sum(lens)
    g = torch.Generator("cuda").manual_seed(13)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    xz, bc, dt = r(T, 2 * D).to(BF), r(T, 2 * N).to(BF), r(T, D).to(BF)
    w, b = (0.5 * r(D, 4)).to(BF), r(D).to(BF)
    A, skip, bias = -torch.rand(D, N, device="cuda", generator=g) - 0.1, r(D), r(D) - 3
    cu = torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)
    x, conv = gdr.causal_conv(xz[:, :D], w, bias=b, cu_seqlens=cu)
    want, bound, last = ref.conv(xz[:, :D], w, b, None, True, lens)
    ref.close(x, want, bound)
    assert torch.equal(ref.wide(conv), last)
    args = dict(D=skip, dt_bias=bias, dt_softplus=True)
    y, h = gdr.selective_scan(x, dt, A, bc[:, :N], bc[:, N:], z=xz[:, D:], cu_seqlens=cu, **args)
    want, bound, end, end_bound = ref.scan(x, dt, A, bc[:, None, :N], bc[:, None, N:], skip, xz[:, D:], bias, True, None, lens)
    ref.close(y, want, bound)
    ref.close(h, end, end_bound)
    for _ in range(steps):
        xz, bc, dt = r(S, 2 * D).to(BF), r(S, 2 * N).to(BF), r(S, D).to(BF)
        before, h0 = conv.clone(), h.clone()
        x = gdr.causal_conv_step(xz[:, :D], w, conv, bias=b)
        want, bound, last = ref.conv(xz[:, None, :D], w, b, before, True)
        ref.close(x, want[:, 0], bound[:, 0])
        assert torch.equal(ref.wide(conv), last)
        y = gdr.selective_scan_step(x, dt, A, bc[:, :N], bc[:, N:], h, z=xz[:, D:], **args)
        one = [t[:, None] for t in (x, dt)] + [A] + [t[:, None, None] for t in (bc[:, :N], bc[:, N:])]
        want, bound, end, end_bound = ref.scan(*one, skip, xz[:, None, D:], bias, True, h0)
        ref.close(y, want[:, 0], bound[:, 0])
        ref.close(h, end, end_bound)

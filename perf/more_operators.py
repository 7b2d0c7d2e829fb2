"""Cases of the operators in front of the recurrence and beside it: the short causal convolution,
the norm and rotation of queries and keys, and the selective scan.

A recurrent layer runs them in this order: ``causal_conv`` over the columns of one projection (q, k
and v out of it as separate tensors, or x), ``qk_norm_rope`` on q and k, then the delta rule; or
``selective_scan`` on x.  Single tokens go through ``causal_conv_step`` and ``selective_scan_step``,
which carry the state (here from one buffer to another, so that a pass leaves its inputs as they
were).  Head shapes are HK = 16, HV = 32, dk = dv = 128: 8192 columns of q, k and v, 4096 channels
of the scan.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
MOST_VALUES = 4097 * 8192         # values convolved in the largest listed case
MOST_STEPS = 32768                # tokens in a row in the longest listed scan
MOST_STATES = 32768 * 4096 * 16   # tokens times state values of it
MOST_CARRIED = 256 * 4096 * 16    # state values of the largest listed step


def listed():
    return [
        # q, k and v of one new token of one sequence: the call's latency
        dict(name="conv_step_1x8192", op="conv_step", rows=1, splits="2048,2048,4096", width=4, dtype="bf16", wdtype="bf16", bias=False, silu=True),
        # a decode step of 32 sequences
        dict(name="conv_step_32x8192", op="conv_step", rows=32, splits="2048,2048,4096", width=4, dtype="bf16", wdtype="bf16", bias=False, silu=True),
        # a prompt of 4097 tokens
        dict(name="conv_4097x8192", op="conv", lens="4097", packed=False, splits="2048,2048,4096", width=4, dtype="bf16", wdtype="bf16", bias=False, silu=True, carried=False),
        # prompts of any length laid end to end (a resumed one, an empty one), nothing a multiple of anything
        dict(name="conv_packed_2999x1001_f32", op="conv", lens="701,1,0,33,1500,2,762", packed=True, splits="333,668", width=3, dtype="f32", wdtype="f32", bias=True, silu=True, carried=True),
        # a decode step of 32 sequences
        dict(name="scan_step_32x4096x16", op="scan_step", rows=32, channels=4096, states=16, groups=1, dtype="bf16", dtdtype="bf16", gate=True),
        # a decode step of a large batch: the state's bytes
        dict(name="scan_step_256x4096x16", op="scan_step", rows=256, channels=4096, states=16, groups=1, dtype="bf16", dtdtype="bf16", gate=True),
        # a prompt of 4097 tokens
        dict(name="scan_4097x4096x16", op="scan", lens="4097", packed=False, channels=4096, states=16, groups=1, dtype="bf16", dtdtype="bf16", gate=True, carried=False),
        # a packed batch of 8 sequences, each continued from a state
        dict(name="scan_packed_4100x4096x16", op="scan", lens="513,97,1024,0,64,1377,1,1024", packed=True, channels=4096, states=16, groups=1, dtype="bf16", dtdtype="bf16", gate=True, carried=True),
        # short sequences, odd sizes, fp32, no gate
        dict(name="scan_3x333x1001x10_f32", op="scan", lens="333,333,333", packed=False, channels=1001, states=10, groups=1, dtype="f32", dtdtype="f32", gate=False, carried=True),
        # a long prompt
        dict(name="scan_32768x4096x16", op="scan", lens="32768", packed=False, channels=4096, states=16, groups=1, dtype="bf16", dtdtype="bf16", gate=True, carried=False),
        # queries and keys of a decode step of 32 sequences
        dict(name="qk_32x16+16x128", op="qk", rows=32, qheads=16, kheads=16, dim=128, rotated=128, pairs="halves", dtype="bf16", wdtype="bf16", length=32768, fused=False),
        # of a prompt of 4097 tokens, as column ranges of one projection's output
        dict(name="qk_4097x32+16x128", op="qk", rows=4097, qheads=32, kheads=16, dim=128, rotated=128, pairs="halves", dtype="bf16", wdtype="bf16", length=4097, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width between lo and hi: a multiple of 64 two times in three, any number otherwise."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 1 / 3 else max(64, n // 64 * 64)


def _lens(rng, most):
    """Lengths of a packed batch: most ordinary ones, some short, some of nothing at all."""
    lens = []
    for _ in range(rng.randint(2, 12)):
        lens.append(rng.choice([0, 1, 2, 3]) if rng.random() < 0.3 else _log(rng, 1, max(1, most // 6)))
    return lens if any(lens) else [5]


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "qk"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_step"):
        cols = _width(rng, 256, 12288)
        splits = [cols]
        if rng.random() < 0.5:
            cut = max(1, int(cols * rng.uniform(0.2, 0.8)))
            cut = cut // 64 * 64 if cols % 64 == 0 and cut >= 64 else cut
            splits = [cut, cols - cut]
        case = dict(op=op, splits=",".join(str(n) for n in splits), width=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    wdtype=rng.choice([dtype, "f32"]), bias=rng.random() < 0.5, silu=rng.random() < 0.8)
        if op == "conv_step":
            return dict(case, rows=_log(rng, 1, 512))
        case["packed"] = rng.random() < 0.5
        most = MOST_VALUES // 2 // cols
        lens = _lens(rng, most) if case["packed"] else [_log(rng, 1, most)]
        if not case["packed"]:
            lens = lens * max(1, min(rng.randint(1, 8), most // lens[0]))
        return dict(case, lens=",".join(str(n) for n in lens), carried=rng.random() < 0.5)
    if op in ("scan", "scan_step"):
        groups = rng.choice([1, 1, 1, 2, 4])
        case = dict(op=op, channels=_width(rng, 64, 4096 // groups) * groups, states=rng.choice([16, 16, 16, 4, 8, 32, 64, rng.randint(1, 40)]),
                    groups=groups, dtype=dtype, dtdtype=rng.choice([dtype, "f32"]), gate=rng.random() < 0.7)
        size = case["channels"] * case["states"]
        if op == "scan_step":
            return dict(case, rows=_log(rng, 1, min(512, MOST_CARRIED // size)))
        case["packed"] = rng.random() < 0.4
        most = min(MOST_STEPS // 4, MOST_STATES // 4 // size)
        lens = _lens(rng, most) if case["packed"] else [_log(rng, 1, most)]
        if not case["packed"]:
            lens = lens * max(1, min(rng.randint(1, 8), MOST_STATES // 4 // (size * lens[0])))
        return dict(case, lens=",".join(str(n) for n in lens), carried=rng.random() < 0.5)
    dim = rng.choice([32, 64, 64, 128, 128, 128, 256, 80, 2 * rng.randint(1, 100)])
    rotated = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
    qheads = rng.choice([1, 4, 7, 8, 16, 32])
    kheads = rng.choice([1, 2, 8, qheads])
    rows = _log(rng, 1, MOST_VALUES // 4 // ((qheads + kheads) * dim))
    return dict(op=op, rows=rows, qheads=qheads, kheads=kheads, dim=dim, rotated=rotated, pairs=rng.choice(["halves", "halves", "neighbours"]),
                dtype=dtype, wdtype=rng.choice([dtype, "f32"]), length=_log(rng, 16, 65536), fused=rng.random() < 0.5)


def _ints(text):
    return [int(n) for n in text.split(",")]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    st = dict(case=case)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op in ("conv", "scan"):
        lens = _ints(case["lens"])
        lead = (sum(lens),) if case["packed"] else (len(lens), lens[0])
        seqs = len(lens)
        st["cu"] = None
        if case["packed"]:
            ends = torch.tensor([0] + lens).cumsum(0)
            st["cu"] = ends.to(torch.int32).cuda()
            st["bounds"] = ends.tolist()
    elif op in ("conv_step", "scan_step"):
        lead, seqs = (case["rows"],), case["rows"]
    if op in ("conv", "conv_step"):
        splits, W = _ints(case["splits"]), case["width"]
        D, wt = sum(splits), DTYPES[case["wdtype"]]
        st["x"] = normal(*lead, D).to(dt)
        st["weight"] = (W ** -0.5 * normal(D, W)).to(wt)
        st["bias"] = (0.1 * normal(D)).to(wt) if case["bias"] else None
        st["state"] = normal(seqs, W - 1, D).to(dt) if case.get("carried", True) else None
        st["splits"] = splits
        st["out"] = [torch.empty(*lead, n, device="cuda", dtype=dt) for n in splits]
        st["out_state"] = torch.empty(seqs, W - 1, D, device="cuda", dtype=dt)
    elif op in ("scan", "scan_step"):
        D, N, G = case["channels"], case["states"], case["groups"]
        x = normal(*lead, D)
        st["x"] = (x * torch.sigmoid(x)).to(dt)             # what the convolution's SiLU leaves
        st["dt"] = (0.5 * normal(*lead, D)).to(DTYPES[case["dtdtype"]])
        step = torch.exp(math.log(1e-3) + uniform(D) * math.log(100.0))
        st["dt_bias"] = torch.log(torch.expm1(step))        # steps of 0.001 to 0.1
        st["A"] = -(torch.arange(1, N + 1, device="cuda") * (0.9 + 0.2 * uniform(D, N)))
        st["B"], st["C"] = normal(*lead, G, N).to(dt), normal(*lead, G, N).to(dt)
        st["D"] = 1.0 + 0.1 * normal(D)
        st["z"] = normal(*lead, D).to(dt) if case["gate"] else None
        st["h0"] = 0.3 * normal(seqs, D, N) if case.get("carried", True) else None
        st["out"] = torch.empty(*lead, D, device="cuda", dtype=dt)
        st["ht"] = torch.empty(seqs, D, N, device="cuda")
    else:
        M, HQ, HK, d = case["rows"], case["qheads"], case["kheads"], case["dim"]
        both = normal(M, HQ + HK, d) * torch.exp(0.5 * normal(M, HQ + HK, 1))
        both = both.to(dt)
        st["q"], st["k"] = both[:, :HQ], both[:, HQ:]       # column ranges of one tensor
        if not case["fused"]:
            st["q"], st["k"] = st["q"].contiguous(), st["k"].contiguous()
        wt = DTYPES[case["wdtype"]]
        st["q_weight"], st["k_weight"] = (1.0 + 0.2 * normal(d)).to(wt), (1.0 + 0.2 * normal(d)).to(wt)
        half, length = case["rotated"] // 2, case["length"]
        speed = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * speed
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        if M == length:                                      # a prompt
            st["positions"] = torch.arange(M, device="cuda", dtype=torch.int32)
        else:                                                # new tokens of many sequences
            st["positions"] = torch.randint(0, length, (M,), device="cuda", dtype=torch.int32, generator=gen)
        st["out_q"] = torch.empty(M, HQ, d, device="cuda", dtype=dt)
        st["out_k"] = torch.empty(M, HK, d, device="cuda", dtype=dt)
    return st


def run(state):
    if own:
        return _kernels(state)
    return {"conv": _conv, "conv_step": _conv_step, "scan": _scan, "scan_step": _scan_step, "qk": _qk}[state["case"]["op"]](state)


def _kernels(st):
    import gated_delta_rule_70_amd as gdr

    case = st["case"]
    op = case["op"]
    if op == "conv":
        return gdr.causal_conv(st["x"], st["weight"], bias=st["bias"], state=st["state"], cu_seqlens=st["cu"],
                               activation="silu" if case["silu"] else None, out=st["out"], out_state=st["out_state"])
    if op == "conv_step":
        return gdr.causal_conv_step(st["x"], st["weight"], st["state"], bias=st["bias"],
                                    activation="silu" if case["silu"] else None, out=st["out"],
                                    out_state=st["out_state"]), st["out_state"]
    if op == "scan":
        return gdr.selective_scan(st["x"], st["dt"], st["A"], st["B"], st["C"], D=st["D"], z=st["z"], dt_bias=st["dt_bias"],
                                  dt_softplus=True, h0=st["h0"], cu_seqlens=st["cu"], out=st["out"], ht=st["ht"])
    if op == "scan_step":
        return gdr.selective_scan_step(st["x"], st["dt"], st["A"], st["B"], st["C"], st["h0"], D=st["D"], z=st["z"],
                                       dt_bias=st["dt_bias"], dt_softplus=True, out=st["out"], out_state=st["ht"]), st["ht"]
    return gdr.qk_norm_rope(st["q"], st["k"], st["q_weight"], st["k_weight"], st["cos"], st["sin"], positions=st["positions"],
                            eps=EPS, interleaved=case["pairs"] == "neighbours", out_q=st["out_q"], out_k=st["out_k"])


def _sequences(st, *names):
    """The sequences one after the other, or a dense batch at once: the named tensors as [B, T, ...],
    and which of the states they go with."""
    if st["cu"] is None:
        yield [None if st[n] is None else st[n] for n in names], slice(None)
        return
    for i, (a, b) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        yield [None if st[n] is None else st[n][None, a:b] for n in names], slice(i, i + 1)


def _conv_rows(x, before, st):
    """x [B, T, D] behind the W - 1 rows ``before``: outputs in fp32, and the last W - 1 rows."""
    W, w = st["case"]["width"], st["weight"].float()
    whole = torch.cat([before, x], 1)
    T = x.shape[1]
    y = whole[:, :T].float() * w[:, 0]
    for j in range(1, W):
        y = y + whole[:, j:j + T].float() * w[:, j]
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if st["case"]["silu"]:
        y = y / (1.0 + torch.exp(-y))
    return y.to(x.dtype), whole[:, T:]


def _conv(st):
    before = torch.zeros_like(st["out_state"]) if st["state"] is None else st["state"]
    ys, ends = [], []
    for (x,), i in _sequences(st, "x"):
        y, end = _conv_rows(x, before[i], st)
        ys.append(y)
        ends.append(end)
    y = ys[0] if st["cu"] is None else torch.cat(ys, 1)[0]
    return tuple(p.contiguous() for p in y.split(st["splits"], dim=-1)), torch.cat(ends).contiguous()


def _conv_step(st):
    y, end = _conv_rows(st["x"][:, None], st["state"], st)
    return tuple(p.contiguous() for p in y[:, 0].split(st["splits"], dim=-1)), end.contiguous()


def _softplus(v):
    # 64 bits: far below zero it is exp(v), which 1 + exp(v) has no bits for
    v = v.double()
    return (torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))).float()


def _scan_rows(x, dt, B, C, z, h, st, block=64):
    """[B, T, ...] from the states h: outputs in x's type, and the states behind them."""
    A, G = st["A"], B.shape[2]
    per = x.shape[2] // G
    ys = []
    for t0 in range(0, x.shape[1], block):
        s = slice(t0, t0 + block)
        step = _softplus(dt[:, s].float() + st["dt_bias"])
        a = torch.exp(step[..., None] * A)
        b = (step * x[:, s].float())[..., None] * B[:, s].float().repeat_interleave(per, dim=2)
        for t in range(b.shape[1]):
            h = h * a[:, t] + b[:, t]
            b[:, t] = h
        y = (b * C[:, s].float().repeat_interleave(per, dim=2)).sum(-1) + st["D"] * x[:, s].float()
        if z is not None:
            g = z[:, s].float()
            y = y * (g / (1.0 + torch.exp(-g)))
        ys.append(y.to(x.dtype))
    return torch.cat(ys, 1) if ys else x.clone(), h


def _scan(st):
    h0 = torch.zeros_like(st["ht"]) if st["h0"] is None else st["h0"]
    ys, ends = [], []
    for (x, dt, B, C, z), i in _sequences(st, "x", "dt", "B", "C", "z"):
        y, h = _scan_rows(x, dt, B, C, z, h0[i], st)
        ys.append(y)
        ends.append(h)
    return (ys[0] if st["cu"] is None else torch.cat(ys, 1)[0]), torch.cat(ends)


def _scan_step(st):
    one = [None if st[n] is None else st[n][:, None] for n in ("x", "dt", "B", "C", "z")]
    y, h = _scan_rows(*one, st["h0"], st)
    return y[:, 0].contiguous(), h


def _qk(st):
    r = st["case"]["rotated"]
    cos, sin = st["cos"][st["positions"]][:, None], st["sin"][st["positions"]][:, None]
    outs = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        v = x.float()
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()
        if st["case"]["pairs"] == "halves":
            a, b = v[..., :r // 2], v[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = v[..., 0:r:2], v[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        outs.append(torch.cat([turned, v[..., r:]], -1).to(x.dtype))
    return tuple(outs)


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("conv", "scan"):
        lens = _ints(case["lens"])
        rows, seqs, carried = sum(lens), len(lens), case["carried"]
    else:
        rows = seqs = case["rows"]
        carried = True
    if op in ("conv", "conv_step"):
        D, W = sum(_ints(case["splits"])), case["width"]
        return {"bytes": 2 * rows * D * e + seqs * (W - 1) * D * e * (2 if carried else 1)
                + D * (W + (1 if case["bias"] else 0)) * BYTES[case["wdtype"]],
                "flops": rows * D * (2 * W + (4 if case["silu"] else 0))}
    if op in ("scan", "scan_step"):
        D, N = case["channels"], case["states"]
        return {"bytes": rows * (D * (e * (3 if case["gate"] else 2) + BYTES[case["dtdtype"]]) + 2 * case["groups"] * N * e)
                + seqs * D * N * 4 * (2 if carried else 1) + 4 * D * (N + 2),
                "flops": rows * D * (7 * N + 8)}
    n = case["rows"] * (case["qheads"] + case["kheads"]) * case["dim"]
    return {"bytes": 2 * n * e + case["rows"] * (4 * case["rotated"] + 4) + 2 * case["dim"] * BYTES[case["wdtype"]], "flops": 8 * n}


def exact(case, seed):
    """The definitions in 64 bits."""
    st = prepare(case, seed)
    wide = {k: v.to(torch.float64) if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}
    if case["op"] in ("conv", "conv_step"):
        return _exact_conv(case, wide)
    if case["op"] in ("scan", "scan_step"):
        return _exact_scan(case, wide)
    outs = []
    r = case["rotated"]
    turn = torch.complex(wide["cos"], wide["sin"]).index_select(0, st["positions"].long()).unsqueeze(1)
    for name in ("q", "k"):
        v = wide[name]
        power = (v * v).sum(-1, keepdim=True) / case["dim"] + EPS
        v = v / power.sqrt() * wide[name + "_weight"]
        head = v[..., :r]
        if case["pairs"] == "halves":
            head = head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
        else:
            head = head.unflatten(-1, (r // 2, 2))
        p = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
        if case["pairs"] == "halves":
            p = p.transpose(-1, -2)
        outs.append(torch.cat([p.flatten(-2), v[..., r:]], -1))
    return tuple(outs)


def _spans(case):
    """(first row, rows) of every sequence, over the rows laid end to end."""
    if case["op"].endswith("step"):
        return [(i, 1) for i in range(case["rows"])]
    spans, at = [], 0
    for n in _ints(case["lens"]):
        spans.append((at, n))
        at += n
    return spans


def _exact_conv(case, st):
    W, D = case["width"], st["weight"].shape[0]
    x = st["x"].reshape(-1, D)
    spans = _spans(case)
    if case["op"] == "conv_step":                 # all rows at once
        rows = torch.cat([st["state"], x.unsqueeze(1)], 1)
        acc = (rows * st["weight"].t()).sum(1)
        ends = rows[:, 1:]
    else:
        acc, ends = torch.zeros_like(x), torch.zeros(len(spans), W - 1, D, dtype=torch.float64, device=x.device)
        for i, (at, n) in enumerate(spans):
            past = ends[i].clone() if st["state"] is None else st["state"][i]
            for back in range(W):                 # the input `back` tokens before
                tap = st["weight"][:, W - 1 - back]
                k = min(back, n)                  # outputs whose input lies before the sequence
                acc[at + k:at + n] += tap * x[at:at + n - k]
                if k:
                    acc[at:at + k] += tap * past[W - 1 - back:W - 1 - back + k]
            ends[i] = torch.cat([past, x[max(at, at + n - W + 1):at + n]])[-(W - 1):]
    if st["bias"] is not None:
        acc = acc + st["bias"]
    if case["silu"]:
        acc = acc * torch.sigmoid(acc)
    shape, outs, at = st["x"].shape[:-1], [], 0
    for n in _ints(case["splits"]):
        outs.append(acc[:, at:at + n].reshape(*shape, n))
        at += n
    return tuple(outs), ends.contiguous()


def _exact_scan(case, st, block=32):
    """Within a block of tokens by doubling: (a, b) of neighbouring runs of tokens are joined."""
    D, N, G = case["channels"], case["states"], case["groups"]
    group = torch.arange(D, device="cuda") // (D // G)
    spans = _spans(case)
    y = torch.empty_like(st["x"]).reshape(-1, D)
    flat = {k: None if st[k] is None else st[k].reshape(-1, *st[k].shape[st["x"].dim() - 1:]) for k in ("x", "dt", "B", "C", "z")}
    h = torch.zeros(len(spans), D, N, dtype=torch.float64, device="cuda") if st["h0"] is None else st["h0"].clone()
    n0 = spans[0][1]
    if all(n == n0 for _, n in spans):            # sequences of one length: all at once
        jobs = [(slice(0, len(spans)), 0, n0, len(spans))]
    else:
        jobs = [(slice(i, i + 1), at, n, 1) for i, (at, n) in enumerate(spans)]
    for which, at, n, many in jobs:
        here = {k: None if v is None else v[at:at + n * many].unflatten(0, (many, n)) if n else None for k, v in flat.items()}
        for t0 in range(0, n, block):
            t1 = min(n, t0 + block)
            cut = {k: None if v is None else v[:, t0:t1] for k, v in here.items()}
            step = torch.nn.functional.softplus(cut["dt"] + st["dt_bias"], threshold=1e9)
            a = (step.unsqueeze(-1) * st["A"]).exp()
            b = (step * cut["x"]).unsqueeze(-1) * cut["B"].index_select(2, group)
            reach = 1
            while reach < t1 - t0:
                b = torch.cat([b[:, :reach], b[:, reach:] + a[:, reach:] * b[:, :-reach]], 1)
                a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
                reach *= 2
            b = b + a * h[which].unsqueeze(1)
            h[which] = b[:, -1]
            o = torch.einsum("btdn,btdn->btd", b, cut["C"].index_select(2, group)) + st["D"] * cut["x"]
            if st["z"] is not None:
                o = o * cut["z"] * torch.sigmoid(cut["z"])
            y[at:at + n * many].unflatten(0, (many, n))[:, t0:t1] = o
    return y.reshape(st["x"].shape), h

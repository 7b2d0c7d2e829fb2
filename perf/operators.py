"""Cases of the 8-bit layer operators: the residual norm that quantises, the int8 matrix product
and the gated head norm that quantises.

A gated delta rule layer in 8 bits runs them in this order: ``add_rmsnorm_i8`` (new residual
stream, int8 activations, a scale for each token), ``matmul_i8`` (q, k, v and the output gate from
one product), the delta rule, ``gated_rmsnorm_i8`` (per value head, times silu(gate), int8 again)
and ``matmul_i8`` (the output projection).  Head shapes are HK = 16 or 32, dk = dv = 128.

Where an operator's result is held in 8 bits, ``run`` returns the values that it stands for,
code times scale, in bf16 (fp32 for an fp32 residual stream).
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
MOST_MACS = 32768 * 4096 * 4096   # matrix product of the largest listed case
MOST_VALUES = 32768 * 4096        # values normed in the largest listed case


def listed():
    return [
        # one new token of one sequence: the call's latency
        dict(name="norm_1x4096", op="norm", rows=1, cols=4096, dtype="bf16", wdtype="bf16", residual=True),
        # a decode step of 32 sequences
        dict(name="norm_32x4096", op="norm", rows=32, cols=4096, dtype="bf16", wdtype="f32", residual=True),
        # a prompt of 4097 tokens
        dict(name="norm_4097x4096", op="norm", rows=4097, cols=4096, dtype="bf16", wdtype="bf16", residual=True),
        # a long prompt, or a packed batch of them
        dict(name="norm_32768x4096", op="norm", rows=32768, cols=4096, dtype="bf16", wdtype="bf16", residual=True),
        # odd width, fp32 stream, first layer (nothing to add yet)
        dict(name="norm_777x1001_f32", op="norm", rows=777, cols=1001, dtype="f32", wdtype="f32", residual=False),
        # outputs of a decode step of 32 sequences (the delta rule's fp32 o)
        dict(name="gated_32x32x128", op="gated", rows=32, heads=32, dv=128, odtype="f32", zdtype="bf16", wdtype="f32"),
        # outputs of a prompt of 4097 tokens, bf16 o
        dict(name="gated_4097x32x128", op="gated", rows=4097, heads=32, dv=128, odtype="bf16", zdtype="bf16", wdtype="bf16"),
        # q, k, v and gate of one new token: the weights' bytes
        dict(name="product_1x12288x4096", op="product", rows=1, inner=4096, splits="2048,2048,4096,4096", odtype="bf16", bias=False),
        # the same for a decode step of 32 sequences
        dict(name="product_32x12288x4096", op="product", rows=32, inner=4096, splits="2048,2048,4096,4096", odtype="bf16", bias=False),
        # the same for a prompt of 4097 tokens
        dict(name="product_4097x12288x4096", op="product", rows=4097, inner=4096, splits="2048,2048,4096,4096", odtype="bf16", bias=False),
        # output projection of a long prompt
        dict(name="product_32768x4096x4096", op="product", rows=32768, inner=4096, splits="4096", odtype="bf16", bias=False),
        # nothing a multiple of anything: gate logits in fp32 with a bias
        dict(name="product_333x1001x2047_f32", op="product", rows=333, inner=2047, splits="1001", odtype="f32", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width between lo and hi: a multiple of 128 two times in three, any number otherwise."""
    n = _log(rng, lo, hi)
    n = n if rng.random() < 1 / 3 else max(128, n // 128 * 128)
    return n + 1 if n == 24 * 128 else n


def draw(rng):
    op = rng.choice(["norm", "gated", "product", "product"])
    if op == "norm":
        cols = _width(rng, 256, 8192)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, rows=_log(rng, 1, MOST_VALUES // 2 // cols), cols=cols, dtype=dtype,
                    wdtype=rng.choice([dtype, "f32"]), residual=rng.random() < 0.8)
    if op == "gated":
        heads, dv = rng.choice([4, 7, 16, 32, 48, 64]), rng.choice([32, 64, 128])
        return dict(op=op, rows=_log(rng, 1, MOST_VALUES // 2 // (heads * dv)), heads=heads, dv=dv,
                    odtype=rng.choice(["bf16", "f32"]), zdtype=rng.choice(["bf16", "bf16", "f32"]),
                    wdtype=rng.choice(["bf16", "f32"]))
    inner, cols = _width(rng, 256, 8192), _width(rng, 256, 12288)
    splits = str(cols)
    if rng.random() < 0.5:  # two tensors
        cut = max(1, int(cols * rng.uniform(0.2, 0.8)))
        cut = cut // 128 * 128 if cols % 128 == 0 and cut >= 128 else cut
        splits = "%d,%d" % (cut, cols - cut)
    return dict(op=op, rows=_log(rng, 1, max(2, min(16384, MOST_MACS // 2 // (inner * cols)))), inner=inner,
                splits=splits, odtype=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.3)


def _codes(rows, cols, gen):
    """int8 rows and fp32 scales, as quantising normally distributed rows gives them."""
    q = torch.empty(rows, cols, device="cuda", dtype=torch.int8)
    s = torch.empty(rows, device="cuda", dtype=torch.float32)
    step = max(1, (1 << 26) // cols)
    for i in range(0, rows, step):
        v = torch.randn(min(step, rows - i), cols, device="cuda", generator=gen)
        v *= torch.rand(v.shape[0], 1, device="cuda", generator=gen) + 0.5
        top = v.abs().amax(1)
        q[i:i + step] = torch.round(v * (127.0 / top)[:, None]).to(torch.int8)
        s[i:i + step] = top / 127.0
    return q, s


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    st = dict(case=case)
    if case["op"] == "norm":
        M, D, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        loud = torch.ones(D, device="cuda")       # a few channels are much louder than the rest
        loud[torch.randint(0, D, (max(1, D // 512),), device="cuda", generator=gen)] = 20.0
        st["x"] = normal(M, D).to(dt)
        st["residual"] = (3.0 * normal(M, D) * loud).to(dt) if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * normal(D)).to(DTYPES[case["wdtype"]])
        st["q"] = torch.empty(M, D, device="cuda", dtype=torch.int8)
        st["scale"] = torch.empty(M, device="cuda")
        st["sum"] = torch.empty(M, D, device="cuda", dtype=dt) if case["residual"] else None
        st["values"] = torch.empty(M, D, device="cuda", dtype=dt)
        if M > 100:
            st["x"][M // 2] = 0                   # a padding row
            if case["residual"]:
                st["residual"][M // 2] = 0
    elif case["op"] == "gated":
        M, H, V = case["rows"], case["heads"], case["dv"]
        st["o"] = (0.1 * normal(M, H, V) * torch.exp(normal(M, H, 1))).to(DTYPES[case["odtype"]])
        st["gate"] = normal(M, H, V).to(DTYPES[case["zdtype"]])
        st["weight"] = (1.0 + 0.2 * normal(V)).to(DTYPES[case["wdtype"]])
        st["q"] = torch.empty(M, H * V, device="cuda", dtype=torch.int8)
        st["scale"] = torch.empty(M, device="cuda")
        st["values"] = torch.empty(M, H * V, device="cuda", dtype=torch.bfloat16)
    else:
        M, K, dt = case["rows"], case["inner"], DTYPES[case["odtype"]]
        splits = [int(n) for n in case["splits"].split(",")]
        st["a"], st["a_scale"] = _codes(M, K, gen)
        st["w"], st["w_scale"] = _codes(sum(splits), K, gen)
        st["w_scale"] *= K ** -0.5
        st["bias"] = normal(sum(splits)) if case["bias"] else None
        st["splits"] = splits
        st["out"] = [torch.empty(M, n, device="cuda", dtype=dt) for n in splits]
    return st


def run(state):
    if own:
        return _kernels(state)
    return {"norm": _norm, "gated": _gated, "product": _product}[state["case"]["op"]](state)


def _kernels(st):
    import gated_delta_rule_70_amd as gdr

    if st["case"]["op"] == "norm":
        gdr.add_rmsnorm_i8(st["x"], st["weight"], residual=st["residual"], eps=EPS, q=st["q"], scale=st["scale"],
                           out_residual=st["sum"])
        return torch.mul(st["q"], st["scale"][:, None], out=st["values"]), st["scale"], st["sum"]
    if st["case"]["op"] == "gated":
        gdr.gated_rmsnorm_i8(st["o"], st["gate"], st["weight"], eps=EPS, q=st["q"], scale=st["scale"])
        return torch.mul(st["q"], st["scale"][:, None], out=st["values"]), st["scale"]
    return gdr.matmul_i8(st["a"], st["a_scale"], st["w"], st["w_scale"], bias=st["bias"], out=st["out"])


def _norm(st):
    x, r, w = st["x"], st["residual"], st["weight"]
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    # 64 bits: whether 127 t / max rounds up or down is decided next to a border
    t = s.double() * w.double()
    top = t.abs().amax(1)
    q = torch.round(t * 127.0 / torch.where(top > 0, top, 1.0)[:, None])
    rho = torch.rsqrt(s.double().square().mean(1) + EPS)
    scale = (top * rho / 127.0).float()
    return (q.float() * scale[:, None]).to(x.dtype), scale, None if r is None else s


def _gated(st):
    o, z, w = st["o"].double(), st["gate"].double(), st["weight"].double()
    n = o * torch.rsqrt(o.square().mean(2, keepdim=True) + EPS) * w * z / (1.0 + torch.exp(-z))
    n = n.reshape(n.shape[0], -1)
    top = n.abs().amax(1)
    q = torch.round(n * 127.0 / torch.where(top > 0, top, 1.0)[:, None])
    scale = (top / 127.0).float()
    return (q.float() * scale[:, None]).to(torch.bfloat16), scale


def _product(st):
    out = (st["a"].float() @ st["w"].float().t()) * st["a_scale"][:, None] * st["w_scale"]
    if st["bias"] is not None:
        out = out + st["bias"]
    return [p.contiguous() for p in out.to(st["out"][0].dtype).split(st["splits"], dim=1)]


def work(case):
    M = case["rows"]
    if case["op"] == "norm":
        D, e = case["cols"], BYTES[case["dtype"]]
        return {"bytes": M * D * (e * (3 if case["residual"] else 1) + 1) + 4 * M + D * BYTES[case["wdtype"]],
                "flops": 8 * M * D}
    if case["op"] == "gated":
        n = M * case["heads"] * case["dv"]
        return {"bytes": n * (BYTES[case["odtype"]] + BYTES[case["zdtype"]] + 1) + 4 * M, "flops": 15 * n}
    N, K = sum(int(n) for n in case["splits"].split(",")), case["inner"]
    return {"bytes": M * K + N * K + M * N * BYTES[case["odtype"]] + 4 * (M + N * (2 if case["bias"] else 1)),
            "flops": 2 * M * N * K}


def exact(case, seed):
    """The definitions in 64 bits, by rows."""
    st = prepare(case, seed)
    if case["op"] == "product":
        wide = st["w"].to(torch.float64)
        rows = []
        for a, sa in zip(st["a"].split(4096), st["a_scale"].split(4096)):
            p = torch.mm(a.to(torch.float64), wide.t())
            p *= sa.to(torch.float64).unsqueeze(1)
            p *= st["w_scale"].to(torch.float64).unsqueeze(0)
            rows.append(p if st["bias"] is None else p + st["bias"].to(torch.float64).unsqueeze(0))
        whole, at, parts = torch.cat(rows), 0, []
        for n in st["splits"]:
            parts.append(whole[:, at:at + n].contiguous())
            at += n
        return parts
    values, scales, sums = [], [], []
    for i in range(0, case["rows"], 2048):
        if case["op"] == "norm":
            v = st["x"][i:i + 2048].to(torch.float64)
            if case["residual"]:  # the stream holds the sum in its own type, and that is what is normed
                v = (v + st["residual"][i:i + 2048].to(torch.float64)).to(DTYPES[case["dtype"]]).to(torch.float64)
                sums.append(v)
            power = (v * v).sum(1) / case["cols"] + EPS
            v = v * st["weight"].to(torch.float64)
            gain = 1.0 / power.sqrt()
        else:
            v = st["o"][i:i + 2048].to(torch.float64)
            z = st["gate"][i:i + 2048].to(torch.float64)
            power = (v * v).sum(2, keepdim=True) / case["dv"] + EPS
            v = (v / power.sqrt() * st["weight"].to(torch.float64) * (z * torch.sigmoid(z))).flatten(1)
            gain = torch.ones(v.shape[0], dtype=torch.float64, device=v.device)
        most = torch.maximum(v.max(1).values, -v.min(1).values)
        code = (v * 127.0 / most.clamp(min=1e-300).unsqueeze(1)).round()
        scale = most * gain / 127.0
        values.append(code * scale.unsqueeze(1))
        scales.append(scale)
    out = [torch.cat(values), torch.cat(scales)]
    if case["op"] == "norm":
        out.append(torch.cat(sums) if sums else None)
    return out

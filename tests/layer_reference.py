"""The operators before and beside the recurrence in 64 bits, on the CPU, and how far fp32 arithmetic with
one rounding of the result may be from that.

Every function returns the exact values for the given inputs and a bound for each, derived from the
formulas: u = 2^-24 is the relative error of one fp32 operation, 2 u of the hardware's exponential and
reciprocal, and half a step of the output type is added at the end (bf16 2^-8, fp32 2^-24).  Bounds are
first-order; what is left out is below u of them, for which 1 % is added.  Results below fp32's
normal range may be flushed: 2^-125.
"""
import torch

U = 2.0 ** -24
FLUSH = 2.0 ** -125
F64 = torch.float64


def wide(t):
    return None if t is None else t.detach().cpu().to(F64)


def rounding(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, bound):
    """Every value within its bound; NaN where the exact value is NaN, infinities equal."""
    got = wide(got)
    assert got.shape == want.shape, (got.shape, want.shape)
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), "NaN in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), "infinities in other places"
    ok = ~nan & ~inf
    off = (got - want).abs()[ok] - bound[ok]
    if off.numel():
        worst = int(off.argmax())
        assert off[worst] <= 0, (f"off by {(got - want).abs()[ok][worst]:.3e}, bound {bound[ok][worst]:.3e}, value "
                                 f"{want[ok][worst]:.6e} at {ok.nonzero()[worst].tolist()}")


def silu(s, err, out):
    """silu(s) and its error, for s within err: |silu'| <= 1.1; the exponential's argument is taken in two
    parts (2 u, and 2 u of the exponential, 2 u of its correction), one addition, a reciprocal, a product.
    For a bf16 output it is one product with log2(e), itself rounded: the exponent is off by 1.3 u of
    itself at most, and e^-s / (1 + e^-s) of that, relative, is left in the result."""
    y = s * torch.sigmoid(s)
    one = 1.3 * U * s.abs() * y.abs() if out == torch.bfloat16 else 0.0
    return y, 1.1 * err + 12 * U * y.abs() + one + FLUSH


def softplus(v, err):
    """softplus(v) and its error: exp(-|v|) to 6 u, e / (2 + e) another 5 u, the polynomial (7 fused
    steps, falling) 3 u, two more operations; the argument's error times the slope (at most 1, and at most the value)."""
    y = torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))
    return y, 16 * U * y + err * torch.minimum(torch.ones_like(y), y) + FLUSH


def conv(x, weight, bias, state, act, lens=None):
    """x [B, T, D] (a packed batch: [T, D] with lens).  Returns y, bound, last rows [B, W - 1, D]."""
    out = x.dtype
    x, weight, bias, state = wide(x), wide(weight), wide(bias), wide(state)
    D, W = weight.shape
    if lens is None:
        seqs = list(x)
    else:
        seqs, at = [], 0
        for n in lens:
            seqs.append(x[at:at + n])
            at += n
    ys, bounds, ends = [], [], []
    for i, rows in enumerate(seqs):
        whole = torch.cat([torch.zeros(W - 1, D, dtype=F64) if state is None else state[i], rows])
        s, mag = torch.zeros_like(rows), torch.zeros_like(rows)
        for j in range(W):
            s = s + weight[:, j] * whole[j:j + rows.shape[0]]
            mag = mag + (weight[:, j] * whole[j:j + rows.shape[0]]).abs()
        if bias is not None:
            s, mag = s + bias, mag + bias.abs()
        err = (W + 1) * U * mag
        if act:
            s, err = silu(s, err, out)
        ys.append(s)
        bounds.append(1.01 * err + rounding(out) * s.abs() + FLUSH)
        ends.append(whole[rows.shape[0]:])
    join = torch.stack if lens is None else torch.cat
    return join(ys), join(bounds), torch.stack(ends)


def qk(x, weight, cos, sin, positions, eps, interleaved):
    """One of q and k: [rows, heads, d]; positions [rows] or None (0, 1, ...)."""
    out = x.dtype
    x, weight, cos, sin = wide(x), wide(weight), wide(cos), wide(sin)
    d = x.shape[-1]
    n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps)
    n = torch.where((x == 0).all(-1, keepdim=True), torch.zeros_like(n), n)  # with eps = 0
    if weight is not None:
        n = n * weight
    err = 4 * U * n.abs()  # the factor's rounding, two products, the scaling of far heads is exact
    y = n.clone()
    if cos is not None:
        half = cos.shape[1]
        pos = torch.arange(x.shape[0]) if positions is None else positions.cpu().long()
        inside = (pos >= 0) & (pos < cos.shape[0])
        c, s = cos[pos.where(inside, 0)][:, None], sin[pos.where(inside, 0)][:, None]
        c, s = (torch.where(inside[:, None, None], t, float("nan")) for t in (c, s))
        i0, i1 = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        a, b = n[..., i0], n[..., i1]
        y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
        err[..., i0] = 7 * U * ((a * c).abs() + (b * s).abs())
        err[..., i1] = 7 * U * ((b * c).abs() + (a * s).abs())
    return y, 1.01 * err + rounding(out) * y.abs() + FLUSH


def scan(x, dt, A, B, C, D, z, dt_bias, softplus_dt, h0, lens=None):
    """x [B, T, D] (packed: [T, D] with lens), B and C with groups.  Returns y, bound, ht, bound of ht.

    The state's error e follows the recurrence itself: e <- a e + a h (|step A| (r + 2 u) + 3 u) + |in| (r + 3
    u) + u |h|, with r the relative error of step: the exponent's error, of its product and of A's factor
    log2(e), the exponential's own; h stands for the sum of the terms' magnitudes."""
    out = x.dtype
    x, dt, A, B, C, D, z, dt_bias, h0 = (wide(t) for t in (x, dt, A, B, C, D, z, dt_bias, h0))
    ch, N = A.shape
    if lens is None:
        spans = [(i, slice(None)) for i in range(x.shape[0])]
        take = lambda t, s: t[s[0]]
    else:
        spans, at = [], 0
        for n in lens:
            spans.append((None, slice(at, at + n)))
            at += n
        take = lambda t, s: t[s[1]]
    per = ch // B.shape[-2]
    ys, bounds, ends, end_bounds = [], [], [], []
    for i, s in enumerate(spans):
        xs, ds, bs, cs = take(x, s), take(dt, s), take(B, s).repeat_interleave(per, -2), take(C, s).repeat_interleave(per, -2)
        h = torch.zeros(ch, N, dtype=F64) if h0 is None else h0[i].clone()
        mag, e = h.abs(), torch.zeros_like(h)
        yo, bo = torch.zeros_like(xs), torch.zeros_like(xs)
        for t in range(xs.shape[0]):
            v = ds[t] if dt_bias is None else ds[t] + dt_bias
            verr = torch.zeros_like(v) if dt_bias is None else U * v.abs()
            step, serr = softplus(v, verr) if softplus_dt else (v, verr)
            rel = torch.where(step == 0, torch.zeros_like(step), serr / step.abs())
            arg = step[:, None] * A
            a = torch.exp(arg)
            inp = (step * xs[t])[:, None] * bs[t]
            e = a * e + a * mag * (arg.abs() * (rel[:, None] + 2 * U) + 3 * U) + inp.abs() * (rel[:, None] + 3 * U)
            h, mag = a * h + inp, a * mag + inp.abs()
            e = e + U * mag + FLUSH
            y, err = (cs[t] * h).sum(-1), (cs[t].abs() * (e + (N + 2) * U * mag)).sum(-1)
            if D is not None:
                y, err = y + D * xs[t], err + 2 * U * (D * xs[t]).abs() + U * y.abs()
            if z is not None:
                zt = take(z, s)[t]
                g, gerr = silu(zt, torch.zeros_like(zt), out)
                y, err = y * g, err * g.abs() + y.abs() * gerr + U * (y * g).abs()
            yo[t], bo[t] = y, 1.01 * err + rounding(out) * y.abs() + FLUSH
        ys.append(yo)
        bounds.append(bo)
        ends.append(h)
        end_bounds.append(1.01 * e + FLUSH)
    join = torch.stack if lens is None else torch.cat
    return join(ys), join(bounds), torch.stack(ends), torch.stack(end_bounds)

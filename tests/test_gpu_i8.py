"""The 8-bit operators against their definitions in 64 bits.

Tolerances, derived from the number of roundings (U = 2^-24, half a step of fp32):
  * the residual stream and the norm's codes are exact (codes of an exact quotient, ties to
    even), its scale is rounded once from fp64: 1.01 U;
  * gated norm: n carries at most 16 U of relative error (rho, four products, the exponential to
    2 U, the sum, the division, the hardware exponent to 2 U), so a code may be off the nearest
    one by what 16 U of 127 steps is, and the scale by 18 U;
  * product: the int32 sum is exact; conversion, two scales: 3 U of the product's magnitude,
    then bias and sum: U of the result; bf16 results half a step more, 2^-8."""
import pytest
import torch

import gated_delta_rule_70_amd as gdr
from gpu_util import note

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def rand(*shape, dtype=F32, seed=0, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def codes(*shape, seed=0, lo=-128):
    return torch.randint(lo, 128, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int8)


def norm_reference(x, w, r, eps):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    t = s.double() * w.double()
    top = t.abs().amax(-1)
    q = torch.round(t * 127.0 / torch.where(top > 0, top, 1.0)[..., None]).nan_to_num(0.0)
    scale = top / torch.sqrt(s.double().square().mean(-1) + eps) / 127.0
    scale = torch.where(top == 0, 0.0, scale)
    bad = ~(top <= 3.402823466e38)
    return s, torch.where(bad[..., None], 0.0, q), torch.where(bad, float("nan"), scale)


def check_norm(x, w, r, eps=1e-6, **kw):
    s, q_ref, scale_ref = norm_reference(x, w, r, eps)
    note(f"add_rmsnorm_i8 x={tuple(x.shape)} {x.dtype} {w.dtype} residual={r is not None}")
    q, scale, out = gdr.add_rmsnorm_i8(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=eps, **kw)
    torch.cuda.synchronize()
    assert (out is None) == (r is None)
    if r is not None:
        assert torch.equal(out.cpu().nan_to_num(7.0), s.nan_to_num(7.0))
    assert torch.equal(q.cpu().double(), q_ref)
    scale = scale.cpu().double()
    assert torch.equal(scale.isnan(), scale_ref.isnan())
    assert bool(((scale - scale_ref).abs() <= 1.01 * U * scale_ref)[~scale_ref.isnan()].all())
    return q, scale


@pytest.mark.parametrize("dtypes", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16_wf32", "f32"])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 511, 512, 513, 1001, 2048, 2056, 4096, 4100, 5120, 8192, 8200, 16384, 32768])
def test_add_rmsnorm(D, dtypes):
    x = rand(5, D, dtype=dtypes[0], seed=D)
    r = rand(5, D, dtype=dtypes[0], seed=D + 1, scale=4.0)
    w = (1 + rand(D, dtype=F32, seed=D + 2, scale=0.3)).to(dtypes[1])
    check_norm(x, w, r)
    check_norm(x[:1], w, None)


@pytest.mark.parametrize("D", [520, 1000, 1001, 1024, 1032, 8192, 8195, 16384])
def test_add_rmsnorm_of_many_rows(D):
    M = 4100 if D < 2000 else 300
    x, r, w = rand(M, D, dtype=BF, seed=D), rand(M, D, dtype=BF, seed=D + 1, scale=4.0), rand(D, dtype=BF, seed=D + 2)
    check_norm(x, w, r)
    check_norm(x.float(), w.float(), None)


@pytest.mark.parametrize("M,H,V", [(2100, 8, 128), (300, 48, 128), (300, 65, 64), (60, 100, 128), (60, 129, 128)])
@pytest.mark.parametrize("types", [(BF, BF, F32), (F32, BF, F32)], ids=["bf16", "f32"])
def test_gated_rmsnorm_widths(M, H, V, types):
    check_gated(rand(M, H, V, dtype=types[0], seed=M), rand(M, H, V, dtype=types[1], seed=M + 1), rand(V, seed=V).to(types[2]))


@pytest.mark.parametrize("D", [96, 100])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_rmsnorm_many_rows_and_ties(D, dtype):
    # small whole numbers: quotients that lie on a border between two codes are frequent
    x = torch.randint(-254, 255, (1003, D), generator=torch.Generator().manual_seed(3)).to(dtype)
    x[:, 0] = 254
    check_norm(x, torch.ones(D, dtype=dtype), None)
    check_norm(x, torch.ones(D), torch.zeros_like(x))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [264, 333])
def test_add_rmsnorm_special_rows(D, dtype):
    x = rand(14, D, dtype=dtype, seed=1)
    big = torch.finfo(dtype).max
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, D - 1] = float("inf")
    x[3, 0] = -float("inf")
    x[4] *= 1e-30
    x[5] = rand(D, dtype=F32, seed=2).mul(1e30).to(dtype)
    x[6] = 0.0
    x[6, 17] = -3.0            # one value
    x[7, 1::2] = 0.0
    x[8] = 1.0                 # all alike
    x[9] = big / 4             # the squares leave fp32's range
    x[10] = torch.finfo(dtype).tiny
    x[11] = rand(D, dtype=F32, seed=5).mul(1e-37).to(dtype)
    w = torch.full((D,), 1.5, dtype=dtype)
    check_norm(x, w, None)
    check_norm(x, w, torch.zeros_like(x), eps=0.0)
    x[1], x[2], x[3] = 1.0, 2.0, 3.0
    r = -x
    check_norm(x, w, r)        # the sum leaves nothing
    w[7] = float("nan")
    check_norm(x, w, None)
    w[7] = 8.0
    x[:, 7] = big              # t beyond fp32's range
    check_norm(x, w, None)


def test_more_rows_than_one_launch_takes():
    M = (1 << 20) + 5
    x, r, w = (torch.randn(M, 8, device="cuda", dtype=BF) for _ in range(3))
    s, q_ref, scale_ref = norm_reference(x, w[0], r, 1e-6)
    note(f"{M} rows")
    q, scale, out = gdr.add_rmsnorm_i8(x, w[0], r)
    assert torch.equal(out, s) and torch.equal(q.double(), q_ref)
    assert bool(((scale - scale_ref).abs() <= 1.01 * U * scale_ref).all())
    o, z = x.view(M, 8).repeat(1, 4).view(M, 1, 32), r.repeat(1, 4).view(M, 1, 32)
    q, scale = gdr.gated_rmsnorm_i8(o, z, torch.ones(32, device="cuda"))
    tail = slice(M - 40, M)
    q2, scale2 = gdr.gated_rmsnorm_i8(o[tail].contiguous(), z[tail].contiguous(), torch.ones(32, device="cuda"))
    assert torch.equal(q[tail], q2) and torch.equal(scale[tail], scale2)


def test_add_rmsnorm_strides_and_in_place():
    base = rand(6, 5, 200, dtype=BF, seed=4)
    r, w = rand(6, 5, 96, dtype=BF, seed=5), rand(96, dtype=BF, seed=6)
    for off in (0, 8, 5):
        x = base[..., off:off + 96]
        s, q_ref, scale_ref = norm_reference(x, w, r, 1e-6)
        wide = base.cuda()
        note(f"strided x, offset {off}")
        q, scale, out = gdr.add_rmsnorm_i8(wide[..., off:off + 96], w.cuda(), r.cuda(), out_residual=wide[..., off:off + 96])
        torch.cuda.synchronize()
        assert torch.equal(q.cpu().double(), q_ref) and torch.equal(out.cpu(), s)
        want = base.clone()
        want[..., off:off + 96] = s
        assert torch.equal(wide.cpu(), want)      # nothing else was written
    rr = r.cuda()
    q2, _, out2 = gdr.add_rmsnorm_i8(x.cuda(), w.cuda(), rr, out_residual=rr)
    assert out2 is rr and torch.equal(rr.cpu(), s) and torch.equal(q2, q)
    one = rand(96, dtype=BF, seed=8)              # every row the same memory
    check_norm(one.expand(4, 96), w, None)
    # misaligned weight and codes
    wc, qc = torch.empty(97, dtype=BF, device="cuda"), torch.empty(4 * 96 + 3, dtype=torch.int8, device="cuda")
    wc[1:] = w.cuda()
    x = rand(4, 96, dtype=BF, seed=9)
    q3, _, _ = gdr.add_rmsnorm_i8(x.cuda(), wc[1:], q=qc[3:].view(4, 96))
    assert torch.equal(q3.cpu().double(), norm_reference(x, w, None, 1e-6)[1])


def test_single_vectors():
    x, w = rand(96, dtype=BF, seed=1), rand(96, dtype=BF, seed=2)
    q, scale, none = gdr.add_rmsnorm_i8(x.cuda(), w.cuda())
    s, q_ref, scale_ref = norm_reference(x, w, None, 1e-6)
    assert q.shape == (96,) and scale.shape == () and none is None and torch.equal(q.cpu().double(), q_ref)
    wq, ws = gdr.quantize_rows_i8(rand(10, 96, seed=3).cuda())
    y = gdr.matmul_i8(q, scale, wq, ws, out_dtype=F32)
    two = gdr.matmul_i8(q, scale, wq, ws, out_dtype=F32, out=(3, 7))
    assert y.shape == (10,) and torch.equal(torch.cat(two), y)
    assert torch.equal(gdr.matmul_i8(q[None], scale[None], wq, ws, out_dtype=F32)[0], y)
    o, z = rand(3, 32, seed=4), rand(3, 32, seed=5)
    g, gs = gdr.gated_rmsnorm_i8(o.cuda(), z.cuda(), torch.ones(32, device="cuda"))
    assert g.shape == (96,) and gs.shape == ()
    g2, gs2 = gdr.gated_rmsnorm_i8(o[None].cuda(), z[None].cuda(), torch.ones(32, device="cuda"))
    assert torch.equal(g, g2[0]) and torch.equal(gs, gs2[0])


@pytest.mark.parametrize("N,K", [(32776, 32), (32776, 1000)])
def test_outputs_past_four_gigabytes(N, K):
    M = 66000
    a, w = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8), codes(N, K, seed=2)
    sa, sw = torch.rand(M, device="cuda") + 0.1, rand(N, seed=3).abs()
    note(f"outputs past 4 GiB, K={K}")
    y = gdr.matmul_i8(a, sa, w.cuda(), sw.cuda())
    for at in (0, 32768, 65533, M - 70):
        rows = slice(at, min(at + 70, M))
        size, ref = product_reference(a[rows].cpu(), sa[rows].cpu(), w, sw, None)
        tol = 3 * U * size + U * (ref.abs() + 4 * U * size)
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert bool(((y[rows].cpu().double() - ref).abs() <= tol).all())


def test_norm_rows_past_four_gigabytes():
    M, D = 560000, 4096
    x = torch.randn(M, D, device="cuda", dtype=BF)
    note("norm of rows past 4 GiB")
    w = rand(D, dtype=BF, seed=1)
    q, scale, s = gdr.add_rmsnorm_i8(x, w.cuda(), residual=x)
    g, gs = gdr.gated_rmsnorm_i8(x.view(M, 32, 128), x.view(M, 32, 128), torch.ones(128, device="cuda"))
    for at in (0, 262144, 524288, M - 9):
        rows = slice(at, at + 9)
        s_ref, q_ref, _ = norm_reference(x[rows].cpu(), w, x[rows].cpu(), 1e-6)
        assert torch.equal(s[rows].cpu(), s_ref) and torch.equal(q[rows].cpu().double(), q_ref)
        g2, gs2 = gdr.gated_rmsnorm_i8(x[rows].view(9, 32, 128), x[rows].view(9, 32, 128), torch.ones(128, device="cuda"))
        assert torch.equal(g[rows], g2) and torch.equal(gs[rows], gs2)


def test_no_rows():
    q, s, out = gdr.add_rmsnorm_i8(torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,) and out.shape == (0, 64)
    q, s = gdr.gated_rmsnorm_i8(*[torch.empty(2, 0, 4, 64, device="cuda")] * 2, torch.ones(64, device="cuda"))
    assert q.shape == (2, 0, 256) and s.shape == (2, 0)
    y = gdr.matmul_i8(q, s, torch.zeros(5, 256, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"))
    assert y.shape == (2, 0, 5)


def gated_reference(o, z, w, eps):
    o, z = o.double(), z.double()
    n = o / torch.sqrt(o.square().mean(-1, keepdim=True) + eps) * w.double() * (z * torch.sigmoid(z))
    n = torch.where(o == 0, 0.0, n).flatten(-2)
    return n, n.abs().amax(-1)


def check_gated(o, z, w, eps=1e-6):
    n, top = gated_reference(o, z, w, eps)
    note(f"gated_rmsnorm_i8 {tuple(o.shape)} {o.dtype} {z.dtype} {w.dtype}")
    q, scale = gdr.gated_rmsnorm_i8(o.cuda(), z.cuda(), w.cuda(), eps=eps)
    torch.cuda.synchronize()
    q, scale = q.cpu().double(), scale.cpu().double()
    bad = ~(top <= 3.402823466e38)     # NaN, infinity, or beyond fp32's range
    assert torch.equal(scale.isnan(), bad) and not q[bad].any()
    q, scale, n, top = q[~bad], scale[~bad], n[~bad], top[~bad]
    assert bool(((scale - top / 127).abs() <= 18 * U * top / 127).all())
    steps = n * 127.0 / torch.where(top > 0, top, 1.0)[..., None]
    assert bool(((q - steps).abs() <= 0.5 + 2 * 127 * 18 * U).all())   # n's error and the maximum's
    assert not q[top == 0].any()


@pytest.mark.parametrize("types", [(F32, BF, F32), (BF, BF, BF), (F32, F32, BF), (BF, F32, F32)],
                         ids=["f32_bf16", "bf16", "f32_f32", "bf16_f32"])
@pytest.mark.parametrize("M,H,V", [(1, 1, 32), (3, 5, 32), (7, 3, 64), (2, 4, 128), (5, 7, 128), (130, 8, 64), (3, 32, 128),
                                   (2, 33, 128), (4, 64, 128), (1, 65, 128), (2, 256, 128), (2, 1024, 32)])
def test_gated_rmsnorm(M, H, V, types):
    o = rand(M, H, V, dtype=types[0], seed=M + H, scale=0.2)
    z = rand(M, H, V, dtype=types[1], seed=M + H + 1, scale=2.0)
    check_gated(o, z, (1 + rand(V, seed=V, scale=0.2)).to(types[2]))


@pytest.mark.parametrize("zt", [BF, F32])
def test_gated_rmsnorm_special_rows(zt):
    o, z, w = rand(12, 6, 64, seed=1), rand(12, 6, 64, seed=2).to(zt), torch.ones(64)
    o[0] = 0.0
    o[1, 2] = 0.0
    o[2, 3, 4] = float("nan")
    z[3, 0, 0] = float("inf")
    z[4, 5, 63] = float("nan")
    o[5] *= 1e-25
    o[6] *= 1e25
    z[7] = -120.0
    z[8] = 120.0
    z[9, 1] = torch.finfo(zt).max / 2
    z[10, 1] = -torch.finfo(zt).max
    o[11, 1] = float("inf")
    z[7] = -60.0
    check_gated(o, z, w)
    check_gated(o, z, w, eps=0.0)
    # silu far out on the negative side
    z = torch.linspace(-85, 85, 6 * 64).view(1, 6, 64).to(zt)
    for i in range(6):
        check_gated(torch.ones(1, 1, 64), z[:, i:i + 1].contiguous(), w)


@pytest.mark.parametrize("ot", [BF, F32])
def test_gated_rmsnorm_heads_below_the_normal_range(ot):
    """Without eps a head's norm is finite however small its values are: one value of fp32's
    smallest ones among normal heads, and rows of nothing else."""
    o, z = rand(4, 6, 64, seed=1).to(ot), rand(4, 6, 64, dtype=BF, seed=2)
    tiny = torch.finfo(ot).smallest_normal / 64
    o[0, 2] = tiny
    o[1] = (rand(6, 64, seed=3).sign() * tiny).to(ot)
    o[2, 1] = 0.0
    o[2, 1, 5] = -tiny
    o[3] = rand(6, 64, seed=4, scale=1e-38).to(ot)
    check_gated(o, z, torch.ones(64), eps=0.0)


def test_gated_rmsnorm_strides():
    wide_o, wide_z = rand(5, 1000, seed=1), rand(5, 900, dtype=BF, seed=2)
    w = rand(32, seed=3)
    for off in (0, 4, 3):
        o, z = wide_o[:, off:off + 224].unflatten(1, (7, 32)), wide_z[:, off + 8:off + 232].unflatten(1, (7, 32))
        q, s = gdr.gated_rmsnorm_i8(wide_o.cuda()[:, off:off + 224].unflatten(1, (7, 32)),
                                    wide_z.cuda()[:, off + 8:off + 232].unflatten(1, (7, 32)), w.cuda())
        q2, s2 = gdr.gated_rmsnorm_i8(o.contiguous().cuda(), z.contiguous().cuda(), w.cuda())
        assert torch.equal(q, q2) and torch.equal(s, s2)


def product_reference(a, sa, w, sw, bias):
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    return p.abs(), p if bias is None else p + bias.double()


def check_product(M, N, K, dtype=BF, bias=False, seed=0, out=None, lo=-128):
    a, w = codes(M, K, seed=seed, lo=lo), codes(N, K, seed=seed + 1, lo=lo)
    sa, sw = rand(M, seed=seed + 2).abs() + 0.1, rand(N, seed=seed + 3).abs() * K ** -0.5
    b = rand(N, seed=seed + 4) if bias else None
    size, ref = product_reference(a, sa, w, sw, b)
    note(f"matmul_i8 M={M} N={N} K={K} {dtype} bias={bias} out={out}")
    y = gdr.matmul_i8(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), bias=None if b is None else b.cuda(), out_dtype=dtype, out=out)
    torch.cuda.synchronize()
    if out is not None:
        assert [t.shape[1] for t in y] == list(out) and all(t.is_contiguous() for t in y)
        y = torch.cat(y, 1)
    assert y.dtype == dtype
    tol = 3 * U * size + U * (ref.abs() + 4 * U * size)
    if dtype == BF:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max())} times the tolerance"


@pytest.mark.parametrize("K", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 1024, 2047])
def test_product_reduction_lengths(K):
    for M, N in ((1, 70), (20, 33), (70, 130), (130, 260)):
        check_product(M, N, K, dtype=F32, seed=K)


@pytest.mark.parametrize("M", [1, 2, 8, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 100, 127, 128, 129, 191, 192,
                               193, 255, 256, 257, 300, 511, 513])
def test_product_rows(M):
    check_product(M, 272, 384, seed=M)
    check_product(M, 129, 200, dtype=F32, bias=True, seed=M)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385, 1000])
def test_product_columns(N):
    check_product(5, N, 320, seed=N)
    check_product(77, N, 144, dtype=F32, bias=True, seed=N)
    check_product(300, N, 256, seed=N)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 1000, 8192), (33, 2048, 2048), (640, 1024, 1024), (1025, 2050, 528),
                                   (2048, 2048, 512), (2100, 4097, 300), (4097, 512, 1040)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_product_larger(M, N, K, dtype):
    check_product(M, N, K, dtype=dtype, bias=dtype == F32, seed=M)


# Sizes that each form of the product takes, with operands that can and cannot be copied straight
# to LDS (K a multiple of 16 or not), whole and partial reductions, and rows and columns that end
# inside a tile.
FORMS = {
    "16x16": [(3, 4100, 4096), (50, 250, 1044), (45, 300, 1001)],
    "32x64": [(33, 2048, 2048), (17, 9000, 1040), (250, 700, 999)],
    "128x64": [(640, 1024, 1024), (650, 1000, 784), (600, 1003, 1001)],
    "128x128, four stages": [(2048, 2048, 512), (1025, 2050, 528), (1500, 2050, 903)],
    "128x128": [(1024, 8192, 1024), (1000, 8190, 1040), (2100, 4097, 1001)],
    "256x256": [(4096, 4096, 1024), (4096, 4000, 1568), (4096, 4001, 1553)],
    "256x256 and a launch for the last rows": [(4101, 4000, 1536), (4097, 12288, 2064)],
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_product_forms(form, dtype):
    for M, N, K in FORMS[form]:
        a, w = codes(M, K, seed=1).cuda(), codes(N, K, seed=2).cuda()
        sa, sw = rand(M, seed=3).abs().cuda() + 0.1, rand(N, seed=4).abs().cuda() * K ** -0.5
        b = rand(N, seed=5).cuda() if dtype == F32 else None
        size, ref = product_reference(a, sa, w, sw, b)   # on the GPU, in fp64
        room = torch.full((M + 2, N), 7.0, dtype=dtype, device="cuda")
        note(f"{form}: M={M} N={N} K={K} {dtype}")
        gdr.matmul_i8(a, sa, w, sw, bias=b, out=room[1:M + 1])
        tol = 3 * U * size + U * (ref.abs() + 4 * U * size)
        if dtype == BF:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert bool(((room[1:M + 1].double() - ref).abs() <= tol).all()), (M, N, K)
        assert bool((room[0] == 7.0).all()) and bool((room[M + 1] == 7.0).all())


# The same where rows begin at whole lines, at multiples of 16, at whole words and anywhere: fragments
# are read in place in the first three, and moved by 0 to 3 bytes in the last.
PLACES = [(1, 12288, (512, 528, 532, 515)), (9, 5000, (1024, 1040, 1044, 1001)), (33, 2048, (2048, 2064, 2068, 2049)),
          (64, 4096, (4096, 4112, 4100, 4099, 1023)), (500, 510, (512, 528, 532, 515)), (250, 700, (512, 528, 532, 515, 510)), (640, 1024, (1024, 1040, 1044, 1001)),
          (1000, 2050, (2048, 2064, 2068, 2049, 514)), (1024, 8192, (1024, 1040, 1044, 1001)), (1486, 7920, (2048, 2064, 2068, 2326)),
          (3000, 4001, (1024, 1040, 1044, 1001, 1003)), (4096, 4001, (2048, 2064, 2068, 2049)),
          (4097, 12288, (4096, 2064, 2068, 2049)), (6023, 2690, (2064, 2068, 2049))]


@pytest.mark.parametrize("M,N,Ks", PLACES, ids=[f"{m}x{n}" for m, n, _ in PLACES])
def test_product_places(M, N, Ks):
    for K in Ks:
        a, w = codes(M, K, seed=1).cuda(), codes(N, K, seed=2).cuda()
        sa, sw = rand(M, seed=3).abs().cuda() + 0.1, rand(N, seed=4).abs().cuda() * K ** -0.5
        size, ref = product_reference(a, sa, w, sw, None)
        note(f"M={M} N={N} K={K}")
        y = gdr.matmul_i8(a, sa, w, sw, out_dtype=F32)
        assert bool(((y.double() - ref).abs() <= 3 * U * size + U * ref.abs()).all()), (M, N, K)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N", [(60, 300), (300, 260), (1300, 2060), (2600, 2100)])
def test_product_moved_fragments(M, N, off):
    """Rows of odd distances that begin `off` bytes behind a whole word, in arrays that end with
    their last byte, and whole stages of the reduction up to it."""
    for K in (256, 512, 385, 20):
        pad = 1 + (K % 2)
        wide_a, wide_w = (codes((n - 1) * (K + pad) + K + off, seed=n).cuda() for n in (M, N))
        a = wide_a[off:].as_strided((M, K), (K + pad, 1))
        w = wide_w[off:].as_strided((N, K), (K + pad, 1))
        sa, sw = rand(M, seed=3).abs().cuda() + 0.1, rand(N, seed=4).abs().cuda()
        size, ref = product_reference(a, sa, w, sw, None)
        note(f"M={M} N={N} K={K} off={off}")
        y = gdr.matmul_i8(a, sa, w, sw, out_dtype=F32)
        assert bool(((y.double() - ref).abs() <= 3 * U * size + U * ref.abs()).all()), (M, N, K)


@pytest.mark.parametrize("stride", [(1 << 24) + 16, (1 << 24) + 4, (1 << 24) + 1])
@pytest.mark.parametrize("M", [40, 150])
def test_product_rows_far_apart(M, stride):
    """Rows further apart than a tile's 2^31 bytes: the forms that address each row by itself."""
    K = 300
    buf = torch.zeros((M - 1) * stride + K, dtype=torch.int8, device="cuda")
    a = buf.as_strided((M, K), (stride, 1))
    a.copy_(codes(M, K, seed=1))
    w = codes(2000, K, seed=2).cuda()
    one, ones = torch.ones(M, device="cuda"), torch.ones(2000, device="cuda")
    note(f"rows far apart M={M} stride={stride}")
    want = a.contiguous().double() @ w.double().t()
    assert torch.equal(gdr.matmul_i8(a, one, w, ones, out_dtype=F32).double(), want)
    assert torch.equal(gdr.matmul_i8(w, ones, a, one, out_dtype=F32).double(), want.t())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out", [(1, 1, 1, 1, 1, 1, 1, 255), (131, 127), (5, 250, 3), (7, 1, 250)])
@pytest.mark.parametrize("M", [90, 700, 2500])
def test_product_outputs_that_end_anywhere(M, out, dtype):
    """Outputs whose rows begin at odd addresses and end inside a store, side by side in one array
    that is written nowhere else."""
    K, N = 192, sum(out)
    a, w = codes(M, K, seed=1).cuda(), codes(N, K, seed=2).cuda()
    sa, sw = rand(M, seed=3).abs().cuda() + 0.1, rand(N, seed=4).abs().cuda()
    room = torch.full((M + 2, N + 3 * len(out) + 2), 7.0, dtype=dtype, device="cuda")
    at, parts = 1, []
    for n in out:
        parts.append(room[1:M + 1, at:at + n])
        at += n + 3
    note(f"M={M} out={out} {dtype}")
    gdr.matmul_i8(a, sa, w, sw, out=parts)
    size, ref = product_reference(a, sa, w, sw, None)
    tol = 3 * U * size + U * (ref.abs() + 4 * U * size)
    if dtype == BF:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((torch.cat(parts, 1).double() - ref).abs() <= tol).all())
    for p in parts:
        p.fill_(7.0)
    assert bool((room == 7.0).all())


@pytest.mark.parametrize("out", [(100, 156), (4, 8, 244), (1, 255), (3, 5, 7, 11, 13, 17, 19, 181), (128, 128), (64, 60, 132)])
@pytest.mark.parametrize("M", [1, 40, 70, 300, 1030])
def test_product_separate_outputs(M, out):
    check_product(M, 256, 256, out=out, seed=M)
    check_product(M, 256, 256, dtype=F32, bias=True, out=out, seed=M)


@pytest.mark.parametrize("M", [3, 100, 600])
def test_product_largest_sums(M):
    # the sum of K products of -128 by -128 comes within 2^14 of 2^31
    K = 131071
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    note(f"largest sums M={M}")
    y = gdr.matmul_i8(a, torch.ones(M, device="cuda"), w, torch.ones(20, device="cuda"), out_dtype=F32)
    want = torch.full((20,), 128.0 * 128 * K)
    want[1] = -128.0 * 127 * K
    assert torch.equal(y.cpu(), want.expand(M, 20))


@pytest.mark.parametrize("M", [1, 20, 90, 300])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 16), (16, 48), (3, 5), (1, 0), (4, 4)])
def test_product_strides(M, off, pad):
    """a and w as column ranges of wider arrays, at any byte offset; outputs as column ranges of
    one array, which is written nowhere else."""
    N, K = 150, 272
    wide_a, wide_w = codes(M, off + K + pad, seed=1), codes(N, off + K + pad, seed=2)
    sa, sw = rand(M, seed=3).abs() + 0.1, rand(N, seed=4).abs()
    size, ref = product_reference(wide_a[:, off:off + K], sa, wide_w[:, off:off + K], sw, None)
    room = torch.full((M, N + 40), 7.0, device="cuda")
    outs = (room[:, 8:108], room[:, 120:170])
    note(f"strided product M={M} off={off} pad={pad}")
    gdr.matmul_i8(wide_a.cuda()[:, off:off + K], sa.cuda(), wide_w.cuda()[:, off:off + K], sw.cuda(), out=outs)
    got = torch.cat([t.cpu() for t in outs], 1).double()
    assert bool(((got - ref).abs() <= 3 * U * size + U * ref.abs()).all())
    room[:, 8:108] = 7.0
    room[:, 120:170] = 7.0
    assert bool((room == 7.0).all())


@pytest.mark.parametrize("M", [1, 70, 300])
def test_product_scales_that_are_not_numbers(M):
    a, w = codes(M, 64, seed=1).cuda(), codes(40, 64, seed=2).cuda()
    sa, sw = torch.ones(M, device="cuda"), torch.ones(40, device="cuda")
    sa[M - 1], sw[3] = float("nan"), float("nan")
    y = gdr.matmul_i8(a, sa, w, sw)
    want = torch.zeros(M, 40, dtype=torch.bool)
    want[M - 1], want[:, 3] = True, True
    assert torch.equal(y.isnan().cpu(), want)


def test_product_long_offsets():
    """Rows whose byte offsets pass 2^31 and 2^32 (a view with long strides into one buffer)."""
    K, stride = 96, 1 << 28
    buf = torch.zeros(17 * stride + K, dtype=torch.int8, device="cuda")
    a = buf.as_strided((18, K), (stride, 1))
    a.copy_(codes(18, K, seed=1))
    w = codes(33, K, seed=2)
    ones = torch.ones(33)
    _, ref = product_reference(a.cpu(), ones[:18], w, ones, None)
    note("long offsets")
    y = gdr.matmul_i8(a, ones[:18].cuda(), w.cuda(), ones.cuda(), out_dtype=F32)
    assert torch.equal(y.cpu().double(), ref)
    wide = codes(70, K, seed=3)
    _, ref = product_reference(wide, torch.ones(70), a.cpu(), ones[:18], None)
    y = gdr.matmul_i8(wide.cuda(), torch.ones(70, device="cuda"), a, ones[:18].cuda(), out_dtype=F32)
    assert torch.equal(y.cpu().double(), ref)
    q, scale, _ = gdr.add_rmsnorm_i8(buf.view(torch.uint8)[:16 * stride].view(F32).as_strided((16, 64), (stride // 4, 1)),
                                     torch.ones(64, device="cuda"))
    assert q.shape == (16, 64) and not scale.isinf().any()


def chain(x, res, nw, w1, s1, w2, s2, hw):
    q8, sc, h = gdr.add_rmsnorm_i8(x, nw, residual=res)
    o, z = gdr.matmul_i8(q8, sc, w1, s1, out=(256, 256))
    q8, sc2 = gdr.gated_rmsnorm_i8(o.view(-1, 4, 64), z.view(-1, 4, 64), hw)
    return h, sc, sc2, gdr.matmul_i8(q8, sc2, w2, s2)


def chain_inputs(M, seed):
    D = 512
    w1, s1 = gdr.quantize_rows_i8(rand(512, D, seed=seed + 2).cuda())
    w2, s2 = gdr.quantize_rows_i8(rand(D, 256, seed=seed + 3).cuda())
    return (rand(M, D, dtype=BF, seed=seed).cuda(), rand(M, D, dtype=BF, seed=seed + 1).cuda(),
            torch.ones(D, dtype=BF, device="cuda"), w1, s1, w2, s2, torch.ones(64, device="cuda"))


@pytest.mark.parametrize("M", [1, 50, 500])
def test_repeatable_and_on_another_stream(M):
    x = chain_inputs(M, 10)
    want = chain(*x)
    again = chain(*x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = chain(*x)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b, c in zip(want, again, there):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("M", [1, 70])
def test_both_ways_into_the_library(M, monkeypatch):
    """Calls with every tensor given go through the extension, others through Python: the same
    results, and each is the way taken."""
    x, res, nw, w1, s1, w2, s2, hw = chain_inputs(M, 30)
    q8, sc, h = torch.empty(M, 512, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty_like(x)
    o, z = (torch.empty(M, 256, dtype=BF, device="cuda") for _ in range(2))
    g8, sc2, y = torch.empty(M, 256, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty_like(x)

    def given():
        gdr.add_rmsnorm_i8(x, nw, residual=res, q=q8, scale=sc, out_residual=h)
        assert gdr.matmul_i8(q8, sc, w1, s1, out=[o, z]) == (o, z)
        gdr.gated_rmsnorm_i8(o.view(-1, 4, 64), z.view(-1, 4, 64), hw, q=g8, scale=sc2)
        assert gdr.matmul_i8(g8, sc2, w2, s2, out=y) is y
        return [t.clone() for t in (h, sc, sc2, y)]

    python = chain(x, res, nw, w1, s1, w2, s2, hw)
    with monkeypatch.context() as m:
        m.setattr(gdr.quantized, "_stream", None)      # the way through Python would raise
        native = given()
    with monkeypatch.context() as m:
        class Never:
            add_rmsnorm = gated_rmsnorm = matmul = staticmethod(lambda *a: None)
        m.setattr(gdr.quantized, "_B", Never)
        slow = given()
    for a, b, c in zip(python, native, slow):
        assert torch.equal(a, b) and torch.equal(a, c)
    # bias, and no residual
    b = torch.ones(512, device="cuda")
    assert torch.equal(gdr.matmul_i8(g8, sc2, w2, s2, bias=b, out=y).clone(), gdr.matmul_i8(g8, sc2, w2, s2, bias=b))
    gdr.add_rmsnorm_i8(x, nw, q=q8, scale=sc)
    q_ref, sc_ref, none = gdr.add_rmsnorm_i8(x, nw)
    assert none is None and torch.equal(q8, q_ref) and torch.equal(sc, sc_ref)
    # an error status comes back as the exception: the codes over the input
    with pytest.raises(gdr.GdrError) as e:
        gdr.add_rmsnorm_i8(x, nw, q=x.view(-1).view(torch.int8)[:M * 512].view(M, 512), scale=sc)
    assert e.value.status == 5
    with pytest.raises(ValueError, match="scale must be"):
        gdr.add_rmsnorm_i8(x, nw, q=q8, scale=torch.empty(M + 1, device="cuda"))


def test_stream_argument():
    """Calls given another stream than the current one, whose inputs are dropped at once."""
    side = torch.cuda.Stream()
    want = chain(*chain_inputs(60, 10))
    for stream in (side, side.cuda_stream):
        x, res, nw, w1, s1, w2, s2, hw = chain_inputs(60, 10)
        side.wait_stream(torch.cuda.current_stream())
        q8, sc, h = gdr.add_rmsnorm_i8(x, nw, residual=res, stream=stream)
        o, z = gdr.matmul_i8(q8, sc, w1, s1, out=(256, 256), stream=stream)
        q8, sc2 = gdr.gated_rmsnorm_i8(o.view(-1, 4, 64), z.view(-1, 4, 64), hw, stream=stream)
        y = gdr.matmul_i8(q8, sc2, w2, s2, stream=stream)
        del x, res, nw, w1, s1, q8, o, z
        for _ in range(8):
            torch.full((60, 512), 99.0, device="cuda")
        side.synchronize()
        assert torch.equal(y, want[3]) and torch.equal(h, want[0])


@pytest.mark.parametrize("M", [1, 50, 500])
def test_graph_replays(M):
    x = chain_inputs(M, 20)
    chain(*x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(*x)
    for i in range(3):
        x[0].copy_(rand(M, 512, dtype=BF, seed=100 + i))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, chain(*x)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()

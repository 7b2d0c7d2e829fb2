// Host entry points of the operators before and beside the recurrence (gdr_layer.h): argument
// validation and kernel launches on the caller's stream.  Every check runs before the first HIP call.
#include "gdr_layer.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "arrays.h"
#include "layer_launch.h"

using namespace gdr;

namespace {

// One tensor of a call, for the checks that all share.
struct Operand {
    const void* p;
    int64_t rows, cols, stride, elt;
    bool required;
    Range range;
};

// Pointers given, aligned to their elements, and within 2^62 bytes.
template <int N>
int check(Operand (&o)[N]) {
    for (Operand& t : o)
        if (!t.p && t.required) return GDR_ERR_NULL;
    for (Operand& t : o)
        if (!aligned(t.p, t.elt)) return GDR_ERR_ALIGN;
    for (Operand& t : o)
        if (!range_of(t.p, t.rows, t.cols, t.stride, t.elt, &t.range)) return GDR_ERR_SHAPE;
    return GDR_OK;
}

bool same(const Operand& a, const Operand& b) { return a.p == b.p && (a.rows == 1 || a.stride == b.stride); }

// The rows of a batch, and whether its sizes can be.
int batch_rows(int32_t B, int32_t T, const int32_t* cu, int64_t* rows) {
    if (B < 0 || T < 0) return GDR_ERR_SHAPE;
    *rows = cu ? T : (int64_t)B * T;
    if (*rows > GDR_LAYER_MAX_ROWS || B > GDR_LAYER_MAX_ROWS || (cu && (B < 1 || B > GDR_VARLEN_MAX_SEQS))) return GDR_ERR_SHAPE;
    return aligned(cu, 4) ? GDR_OK : GDR_ERR_ALIGN;
}

int scan_rows(const gdr_scan_dims& d, const int32_t* cu, int64_t* rows) {
    const int st = batch_rows(d.B, d.T, cu, rows);
    if (st != GDR_OK) return st;
    return d.D < 1 || d.D > GDR_LAYER_MAX_CHANNELS || d.N < 1 || d.G < 1 || d.D % d.G ? GDR_ERR_SHAPE : GDR_OK;
}

// Values of workspace.
int64_t scan_workspace(const gdr_scan_dims& d, const ScanCut& cut) {
    return cut.segs > 1 ? (int64_t)d.B * cut.segs * d.D * (d.N + 1) : 0;
}

int scan(const gdr_scan_dims* dims, const int32_t* cu, bool step, const void* x, const void* dt, const float* A,
         const void* B, const void* C, const float* skip, const void* z, const float* dt_bias, const float* h0,
         void* out, float* ht, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dims) return GDR_ERR_NULL;
    const gdr_scan_dims& d = *dims;
    int64_t rows;
    const int st = scan_rows(d, cu, &rows);
    if (st != GDR_OK) return st;
    if (step && d.T != 1) return GDR_ERR_SHAPE;
    if (d.N > GDR_SCAN_MAX_STATES || !known_dtype(d.dtype) || (d.flags & ~GDR_SCAN_DT_SOFTPLUS) ||
        (d.dt_dtype != d.dtype && d.dt_dtype != GDR_F32))
        return GDR_ERR_UNSUPPORTED;
    if (d.x_stride < 0 || d.dt_stride < 0 || d.b_stride < 0 || d.c_stride < 0 || (z && d.z_stride < 0) ||
        (rows > 1 && d.out_stride < d.D))
        return GDR_ERR_SHAPE;
    if (d.B == 0) return GDR_OK;
    const int64_t e = elt_of(d.dtype), some = rows > 0, gn = (int64_t)d.G * d.N, dn = (int64_t)d.D * d.N;
    const ScanCut cut = step || rows == 0 ? ScanCut{1, 0} : scan_cut(d.B, d.T, d.D, d.G, d.N, cu != nullptr);
    const int64_t need = scan_workspace(d, cut);
    enum { X, DT, BB, CC, Z, AA, SKIP, BIAS, H0, OUT, HT, CU, WORK };
    Operand o[] = {{x, rows, d.D, d.x_stride, e, some != 0, {}},
                   {dt, rows, d.D, d.dt_stride, elt_of(d.dt_dtype), some != 0, {}},
                   {B, rows, gn, d.b_stride, e, some != 0, {}},
                   {C, rows, gn, d.c_stride, e, some != 0, {}},
                   {z, rows, d.D, d.z_stride, e, false, {}},
                   {A, d.D, d.N, d.N, 4, some != 0, {}},
                   {skip, 1, d.D, 0, 4, false, {}},
                   {dt_bias, 1, d.D, 0, 4, false, {}},
                   {h0, d.B, dn, dn, 4, false, {}},
                   {out, rows, d.D, d.out_stride, e, some != 0, {}},
                   {ht, d.B, dn, dn, 4, false, {}},
                   {cu, 1, (int64_t)d.B + 1, 0, 4, false, {}},
                   {need ? workspace : nullptr, 1, need, 0, 4, false, {}}};
    const int bad = check(o);
    if (bad != GDR_OK) return bad;
    if (need && (!workspace || workspace_bytes / 4 < (uint64_t)need)) return GDR_ERR_WORKSPACE;
    for (int i = X; i < WORK; ++i)
        if (overlap(o[WORK].range, o[i].range)) return GDR_ERR_ALIAS;
    for (int i : {X, DT, BB, CC, Z, AA, SKIP, BIAS, CU})
        if (overlap(o[OUT].range, o[i].range) || overlap(o[HT].range, o[i].range)) return GDR_ERR_ALIAS;
    if (overlap(o[OUT].range, o[H0].range) || overlap(o[OUT].range, o[HT].range)) return GDR_ERR_ALIAS;
    if (overlap(o[HT].range, o[H0].range) && ht != h0) return GDR_ERR_ALIAS;
    if (rows == 0 && !ht) return GDR_OK;
    ScanArgs a{};
    a.B = d.B, a.T = d.T, a.D = d.D, a.N = d.N, a.G = d.G;
    a.bf16 = d.dtype == GDR_BF16;
    a.dt_bf16 = d.dt_dtype == GDR_BF16;
    a.softplus = d.flags & GDR_SCAN_DT_SOFTPLUS;
    a.x_stride = d.x_stride, a.dt_stride = d.dt_stride, a.z_stride = d.z_stride;
    a.b_stride = d.b_stride, a.c_stride = d.c_stride, a.out_stride = d.out_stride;
    a.cu = cu;
    a.x = x, a.dt = dt, a.z = z, a.b = B, a.c = C;
    a.A = A, a.skip = skip, a.dt_bias = dt_bias, a.h0 = h0;
    a.out = out;
    a.ht = ht;
    a.segs = cut.segs, a.seg_len = cut.seg_len;
    a.workspace = static_cast<float*>(workspace);
    a.stream = static_cast<hipStream_t>(stream);
    return (step ? launch_selective_scan_step(a) : launch_selective_scan(a)) == hipSuccess ? GDR_OK : GDR_ERR_HIP;
}

}  // namespace

extern "C" {

int gdr_causal_conv(const gdr_conv_dims* dims, const int32_t* cu_seqlens, const void* x, const void* weight,
                    const void* bias, const void* state, void* const* outs, void* out_state, void* stream) {
    if (!dims) return GDR_ERR_NULL;
    const gdr_conv_dims& d = *dims;
    int64_t rows;
    const int st = batch_rows(d.B, d.T, cu_seqlens, &rows);
    if (st != GDR_OK) return st;
    if (d.D < 1 || d.D > GDR_LAYER_MAX_CHANNELS || d.W < 1 || d.n_out < 1 || d.n_out > GDR_CONV_MAX_OUT ||
        d.x_stride < 0)
        return GDR_ERR_SHAPE;
    if (d.W < 2 || d.W > 4 || !known_dtype(d.dtype) || (d.flags & ~GDR_CONV_SILU) ||
        (d.weight_dtype != d.dtype && d.weight_dtype != GDR_F32))
        return GDR_ERR_UNSUPPORTED;
    ConvArgs a{};
    int64_t D = 0;
    for (int i = 0; i < d.n_out; ++i) {
        if (d.out_cols[i] < 1 || (rows > 1 && d.out_stride[i] < d.out_cols[i])) return GDR_ERR_SHAPE;
        a.begin[i] = (int)D;
        D += d.out_cols[i];
        if (D > d.D) return GDR_ERR_SHAPE;
    }
    if (D != d.D) return GDR_ERR_SHAPE;
    for (int i = d.n_out; i <= GDR_CONV_MAX_OUT; ++i) a.begin[i] = (int)D;
    if (d.B == 0) return GDR_OK;
    const bool some = rows > 0;
    if (some && !outs) return GDR_ERR_NULL;
    const int64_t e = elt_of(d.dtype), ew = elt_of(d.weight_dtype), tail = (int64_t)(d.W - 1) * D;
    enum { X, W, BIAS, STATE, CU, END };
    Operand o[] = {{x, rows, D, d.x_stride, e, some, {}},
                   {weight, 1, D * d.W, 0, ew, some, {}},
                   {bias, 1, D, 0, ew, false, {}},
                   {state, d.B, tail, tail, e, false, {}},
                   {cu_seqlens, 1, (int64_t)d.B + 1, 0, 4, false, {}},
                   {out_state, d.B, tail, tail, e, false, {}}};
    const int bad = check(o);
    if (bad != GDR_OK) return bad;
    Range out[GDR_CONV_MAX_OUT] = {};
    for (int i = 0; some && i < d.n_out; ++i) {
        if (!outs[i]) return GDR_ERR_NULL;
        if (!aligned(outs[i], e)) return GDR_ERR_ALIGN;
        if (!range_of(outs[i], rows, d.out_cols[i], d.out_stride[i], e, &out[i])) return GDR_ERR_SHAPE;
        for (const Operand& t : o)
            if (overlap(out[i], t.range)) return GDR_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GDR_ERR_ALIAS;
        a.out[i] = outs[i];
        a.out_stride[i] = d.out_stride[i];
    }
    for (int i : {X, W, BIAS, CU})
        if (overlap(o[END].range, o[i].range)) return GDR_ERR_ALIAS;
    if (overlap(o[END].range, o[STATE].range) && out_state != state) return GDR_ERR_ALIAS;
    if (!some && !out_state) return GDR_OK;
    a.B = d.B, a.T = d.T, a.D = d.D, a.W = d.W;
    a.rows = (int)rows;
    a.bf16 = d.dtype == GDR_BF16;
    a.w_bf16 = d.weight_dtype == GDR_BF16;
    a.silu = d.flags & GDR_CONV_SILU;
    a.n_out = d.n_out;
    a.x_stride = d.x_stride;
    a.cu = cu_seqlens;
    a.x = x, a.w = weight, a.bias = bias, a.state = state;
    a.out_state = out_state;
    a.stream = static_cast<hipStream_t>(stream);
    return launch_causal_conv(a) == hipSuccess ? GDR_OK : GDR_ERR_HIP;
}

int gdr_qk_norm_rope(const gdr_qk_dims* dims, const void* q, const void* k, const void* q_weight,
                     const void* k_weight, const float* cos, const float* sin, const void* positions, void* out_q,
                     void* out_k, void* stream) {
    if (!dims) return GDR_ERR_NULL;
    const gdr_qk_dims& d = *dims;
    if (d.rows < 0 || d.rows > GDR_LAYER_MAX_ROWS || d.q_heads < 1 || d.k_heads < 1 || d.q_heads > 65536 ||
        d.k_heads > 65536 || d.dim < 1 || d.rotated < 0 || d.rotated > d.dim || d.rotated % 2 || d.q_stride < 0 ||
        d.k_stride < 0)
        return GDR_ERR_SHAPE;
    if (d.rotated > 0 && (d.table_rows < 1 || (!positions && d.period < 1))) return GDR_ERR_SHAPE;
    if (d.dim > GDR_QK_MAX_DIM || !known_dtype(d.dtype) || (d.flags & ~GDR_QK_INTERLEAVED) ||
        (d.weight_dtype != d.dtype && d.weight_dtype != GDR_F32) ||
        (positions && d.position_bits != 32 && d.position_bits != 64) || !(d.eps >= 0.f) || !std::isfinite(d.eps))
        return GDR_ERR_UNSUPPORTED;
    const int64_t nq = (int64_t)d.q_heads * d.dim, nk = (int64_t)d.k_heads * d.dim;
    if (d.rows > 1 && (d.out_q_stride < nq || d.out_k_stride < nk)) return GDR_ERR_SHAPE;
    if (d.rows == 0) return GDR_OK;
    const int64_t e = elt_of(d.dtype), ew = elt_of(d.weight_dtype), half = d.rotated / 2;
    const bool turn = d.rotated > 0;
    enum { Q, K, OQ, OK };
    Operand o[] = {{q, d.rows, nq, d.q_stride, e, true, {}},
                   {k, d.rows, nk, d.k_stride, e, true, {}},
                   {out_q, d.rows, nq, d.out_q_stride, e, true, {}},
                   {out_k, d.rows, nk, d.out_k_stride, e, true, {}},
                   {q_weight, 1, d.dim, 0, ew, false, {}},
                   {k_weight, 1, d.dim, 0, ew, false, {}},
                   {turn ? cos : nullptr, 1, d.table_rows * half, 0, 4, turn, {}},
                   {turn ? sin : nullptr, 1, d.table_rows * half, 0, 4, turn, {}},
                   {turn ? positions : nullptr, 1, d.rows, 0, d.position_bits == 64 ? 8 : 4, false, {}}};
    const int bad = check(o);
    if (bad != GDR_OK) return bad;
    for (int i : {OQ, OK})
        for (const Operand& t : o) {
            if (&t == &o[i] || (&t == &o[i - OQ] && same(t, o[i]))) continue;
            if (overlap(o[i].range, t.range)) return GDR_ERR_ALIAS;
        }
    QkArgs a{};
    a.rows = d.rows;
    a.heads[0] = d.q_heads, a.heads[1] = d.k_heads;
    a.dim = d.dim, a.rotated = d.rotated, a.table_rows = d.table_rows, a.period = d.period;
    a.bf16 = d.dtype == GDR_BF16;
    a.w_bf16 = d.weight_dtype == GDR_BF16;
    a.interleaved = d.flags & GDR_QK_INTERLEAVED;
    a.wide_positions = d.position_bits == 64;
    a.eps = d.eps;
    a.stride[0] = d.q_stride, a.stride[1] = d.k_stride;
    a.out_stride[0] = d.out_q_stride, a.out_stride[1] = d.out_k_stride;
    a.in[0] = q, a.in[1] = k;
    a.weight[0] = q_weight, a.weight[1] = k_weight;
    a.out[0] = out_q, a.out[1] = out_k;
    a.cos = cos, a.sin = sin;
    a.positions = positions;
    a.stream = static_cast<hipStream_t>(stream);
    return launch_qk_norm_rope(a) == hipSuccess ? GDR_OK : GDR_ERR_HIP;
}

size_t gdr_selective_scan_workspace_bytes(const gdr_scan_dims* dims, int packed) {
    int64_t rows;
    static const int32_t some = 0;
    if (!dims || scan_rows(*dims, packed ? &some : nullptr, &rows) != GDR_OK || dims->N > GDR_SCAN_MAX_STATES || rows == 0) return 0;
    return 4 * static_cast<size_t>(scan_workspace(*dims, scan_cut(dims->B, dims->T, dims->D, dims->G, dims->N, packed != 0)));
}

int gdr_selective_scan(const gdr_scan_dims* dims, const int32_t* cu_seqlens, const void* x, const void* dt,
                       const float* A, const void* B, const void* C, const float* Dskip, const void* z,
                       const float* dt_bias, const float* h0, void* out, float* ht, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return scan(dims, cu_seqlens, false, x, dt, A, B, C, Dskip, z, dt_bias, h0, out, ht, workspace, workspace_bytes, stream);
}

int gdr_selective_scan_step(const gdr_scan_dims* dims, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const float* Dskip, const void* z, const float* dt_bias,
                            const float* h0, void* out, float* ht, void* stream) {
    return scan(dims, nullptr, true, x, dt, A, B, C, Dskip, z, dt_bias, h0, out, ht, nullptr, 0, stream);
}

}  // extern "C"

// Host entry points of the 8-bit operators (gdr_i8.h): argument validation and kernel
// launches on the caller's stream.  Every check runs before the first HIP call.
#include "gdr_i8.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "i8_launch.h"

namespace {

// The bytes of an array of evenly spaced rows.
struct Range {
    uintptr_t lo, hi;        // [lo, hi), from the first value to the last
    uintptr_t width, apart;  // of a row, and from one to the next (0: one row)
};

// The array of `rows` rows of `cols` values, `stride` apart.  False where that passes 2^62.
bool range_of(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t elt, Range* r) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    *r = Range{lo, lo, 0, 0};
    if (!p || rows < 1) return true;
    constexpr int64_t lim = int64_t(1) << 62;
    if (rows > 1 && stride > (lim / elt - cols) / (rows - 1)) return false;
    r->hi = lo + static_cast<uintptr_t>(((rows - 1) * stride + cols) * elt);
    r->width = static_cast<uintptr_t>(cols * elt);
    r->apart = rows > 1 ? static_cast<uintptr_t>(stride * elt) : 0;
    return r->hi >= lo;
}

// Whether two arrays share bytes.  Those with rows equally far apart may be column ranges of one wider
// array, one array's rows between the other's; of any others that cross, it is taken that they do.
bool overlap(const Range& a, const Range& b) {
    if (!(a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi)) return false;
    if (a.apart == 0 || a.apart != b.apart) return true;
    const Range &first = a.lo < b.lo ? a : b, &second = a.lo < b.lo ? b : a;
    const uintptr_t at = (second.lo - first.lo) % a.apart;  // where second's rows begin, from first's
    return at < first.width || second.width > a.apart - at;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool known_dtype(int32_t t) { return t == GDR_BF16 || t == GDR_F32; }

int64_t elt_of(int32_t t) { return t == GDR_F32 ? 4 : 2; }

// The checks that both norms share, on dims alone.
int validate_norm(const gdr_norm_dims* d) {
    if (!d) return GDR_ERR_NULL;
    if (d->rows < 0 || d->rows > GDR_I8_MAX_ROWS || d->heads < 1 || d->cols < 1) return GDR_ERR_SHAPE;
    if ((int64_t)d->heads * d->cols > GDR_NORM_MAX_COLS) return GDR_ERR_SHAPE;
    if (!known_dtype(d->x_dtype) || !known_dtype(d->weight_dtype)) return GDR_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return GDR_ERR_UNSUPPORTED;
    if (d->x_stride < 0) return GDR_ERR_SHAPE;
    return GDR_OK;
}

gdr::NormArgs norm_args(const gdr_norm_dims* d, const void* x, const void* r, const void* w, int8_t* q,
                        float* scale, void* out, void* stream) {
    gdr::NormArgs a{};
    a.rows = d->rows;
    a.heads = d->heads;
    a.cols = d->cols;
    a.x_bf16 = d->x_dtype == GDR_BF16;
    a.gate_bf16 = d->gate_dtype == GDR_BF16;
    a.w_bf16 = d->weight_dtype == GDR_BF16;
    a.eps = d->eps;
    a.x_stride = d->x_stride;
    a.r_stride = d->r_stride;
    a.out_stride = d->out_stride;
    a.x = x;
    a.r = r;
    a.w = w;
    a.q = q;
    a.scale = scale;
    a.out = out;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

}  // namespace

extern "C" {

int gdr_add_rmsnorm_i8(const gdr_norm_dims* dims, const void* x, const void* residual, const void* weight,
                       int8_t* q, float* scale, void* out_residual, void* stream) {
    const int st = validate_norm(dims);
    if (st != GDR_OK) return st;
    const gdr_norm_dims& d = *dims;
    if (d.heads != 1 || (residual && d.r_stride < 0) || (out_residual && d.rows > 1 && d.out_stride < d.cols))
        return GDR_ERR_SHAPE;
    if (d.x_dtype == GDR_F32 && d.weight_dtype != GDR_F32) return GDR_ERR_UNSUPPORTED;
    if (d.rows == 0) return GDR_OK;
    if (!x || !weight || !q || !scale) return GDR_ERR_NULL;
    const int64_t ex = elt_of(d.x_dtype), ew = elt_of(d.weight_dtype);
    if (!aligned(x, ex) || !aligned(residual, ex) || !aligned(out_residual, ex) || !aligned(weight, ew) ||
        !aligned(scale, 4))
        return GDR_ERR_ALIGN;
    Range rx, rr, rw, rq, rs, ro;
    if (!range_of(x, d.rows, d.cols, d.x_stride, ex, &rx) || !range_of(residual, d.rows, d.cols, d.r_stride, ex, &rr) ||
        !range_of(weight, 1, d.cols, 0, ew, &rw) || !range_of(q, d.rows, d.cols, d.cols, 1, &rq) ||
        !range_of(scale, d.rows, 1, 1, 4, &rs) || !range_of(out_residual, d.rows, d.cols, d.out_stride, ex, &ro))
        return GDR_ERR_SHAPE;
    const Range ins[] = {rx, rr, rw};
    for (const Range& r : ins)
        if (overlap(rq, r) || overlap(rs, r)) return GDR_ERR_ALIAS;
    if (overlap(rq, rs) || overlap(rq, ro) || overlap(rs, ro) || overlap(ro, rw)) return GDR_ERR_ALIAS;
    // the new residual stream may replace x or the old one, row for row
    if (overlap(ro, rx) && !(out_residual == x && (d.rows == 1 || d.out_stride == d.x_stride))) return GDR_ERR_ALIAS;
    if (overlap(ro, rr) && !(out_residual == residual && (d.rows == 1 || d.out_stride == d.r_stride)))
        return GDR_ERR_ALIAS;
    gdr::NormArgs a = norm_args(dims, x, residual, weight, q, scale, out_residual, stream);
    a.heads = 0;
    return gdr::launch_add_rmsnorm_i8(a) == hipSuccess ? GDR_OK : GDR_ERR_HIP;
}

int gdr_gated_rmsnorm_i8(const gdr_norm_dims* dims, const void* o, const void* gate, const void* weight,
                         int8_t* q, float* scale, void* stream) {
    const int st = validate_norm(dims);
    if (st != GDR_OK) return st;
    const gdr_norm_dims& d = *dims;
    if (d.r_stride < 0) return GDR_ERR_SHAPE;
    if ((d.cols != 32 && d.cols != 64 && d.cols != 128) || !known_dtype(d.gate_dtype)) return GDR_ERR_UNSUPPORTED;
    if (d.rows == 0) return GDR_OK;
    if (!o || !gate || !weight || !q || !scale) return GDR_ERR_NULL;
    const int64_t eo = elt_of(d.x_dtype), eg = elt_of(d.gate_dtype), ew = elt_of(d.weight_dtype);
    if (!aligned(o, eo) || !aligned(gate, eg) || !aligned(weight, ew) || !aligned(scale, 4)) return GDR_ERR_ALIGN;
    const int64_t n = (int64_t)d.heads * d.cols;
    Range ro, rg, rw, rq, rs;
    if (!range_of(o, d.rows, n, d.x_stride, eo, &ro) || !range_of(gate, d.rows, n, d.r_stride, eg, &rg) ||
        !range_of(weight, 1, d.cols, 0, ew, &rw) || !range_of(q, d.rows, n, n, 1, &rq) ||
        !range_of(scale, d.rows, 1, 1, 4, &rs))
        return GDR_ERR_SHAPE;
    const Range ins[] = {ro, rg, rw};
    for (const Range& r : ins)
        if (overlap(rq, r) || overlap(rs, r)) return GDR_ERR_ALIAS;
    if (overlap(rq, rs)) return GDR_ERR_ALIAS;
    const gdr::NormArgs a = norm_args(dims, o, gate, weight, q, scale, nullptr, stream);
    return gdr::launch_gated_rmsnorm_i8(a) == hipSuccess ? GDR_OK : GDR_ERR_HIP;
}

int gdr_matmul_i8(const gdr_matmul_i8_dims* dims, const int8_t* a, const float* a_scale, const int8_t* w,
                  const float* w_scale, const float* bias, void* const* outs, void* stream) {
    if (!dims) return GDR_ERR_NULL;
    const gdr_matmul_i8_dims& d = *dims;
    if (d.M < 0 || d.M > GDR_I8_MAX_ROWS || d.K < 1 || d.K > GDR_MATMUL_I8_MAX_K || d.n_out < 1 || d.n_out > GDR_MATMUL_I8_MAX_OUT ||
        d.a_stride < 0 || d.w_stride < 0)
        return GDR_ERR_SHAPE;
    if (!known_dtype(d.out_dtype)) return GDR_ERR_UNSUPPORTED;
    const int64_t eo = elt_of(d.out_dtype);
    gdr::MatmulArgs g{};
    int64_t N = 0;
    g.out.n = d.n_out;
    for (int i = 0; i < d.n_out; ++i) {
        if (d.out_cols[i] < 1 || (d.M > 1 && d.out_stride[i] < d.out_cols[i])) return GDR_ERR_SHAPE;
        g.out.begin[i] = (int)N;
        N += d.out_cols[i];
        if (N > (1 << 30)) return GDR_ERR_SHAPE;
    }
    for (int i = d.n_out; i <= GDR_MATMUL_I8_MAX_OUT; ++i) g.out.begin[i] = (int)N;
    // a launch has fewer than 2^32 threads: 2^23 tiles of 256 x 256 with 512 each
    if ((d.M + 255LL) / 256 * ((N + 255) / 256) >= (1LL << 23)) return GDR_ERR_SHAPE;
    if (d.M == 0) return GDR_OK;
    if (!a || !a_scale || !w || !w_scale || !outs) return GDR_ERR_NULL;
    for (int i = 0; i < d.n_out; ++i)
        if (!outs[i]) return GDR_ERR_NULL;
    if (!aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4)) return GDR_ERR_ALIGN;
    Range in[5], out[GDR_MATMUL_I8_MAX_OUT];
    if (!range_of(a, d.M, d.K, d.a_stride, 1, &in[0]) || !range_of(w, N, d.K, d.w_stride, 1, &in[1]) ||
        !range_of(a_scale, d.M, 1, 1, 4, &in[2]) || !range_of(w_scale, N, 1, 1, 4, &in[3]) ||
        !range_of(bias, N, 1, 1, 4, &in[4]))
        return GDR_ERR_SHAPE;
    for (int i = 0; i < d.n_out; ++i) {
        if (!aligned(outs[i], eo)) return GDR_ERR_ALIGN;
        if (!range_of(outs[i], d.M, d.out_cols[i], d.out_stride[i], eo, &out[i])) return GDR_ERR_SHAPE;
        for (const Range& r : in)
            if (overlap(out[i], r)) return GDR_ERR_ALIAS;
        g.out.ptr[i] = outs[i];
        g.out.stride[i] = d.out_stride[i];
    }
    for (int i = 0; i < d.n_out; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GDR_ERR_ALIAS;
    g.M = d.M;
    g.N = (int)N;
    g.K = d.K;
    g.out_bf16 = d.out_dtype == GDR_BF16;
    g.a_stride = d.a_stride;
    g.w_stride = d.w_stride;
    g.a = a;
    g.w = w;
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.bias = bias;
    g.stream = static_cast<hipStream_t>(stream);
    return gdr::launch_matmul_i8(g) == hipSuccess ? GDR_OK : GDR_ERR_HIP;
}

}  // extern "C"

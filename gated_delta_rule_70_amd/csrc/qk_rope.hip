// Root-mean-square norm of query and key heads with the rotation by position (gdr_qk_norm_rope).
#include "layer_launch.h"

#include "row_device.h"

namespace gdr {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(v); }

// The row of the tables that a row of q and k takes, or -1.
__device__ __forceinline__ int table_row(const QkArgs& a, int row) {
    int64_t p = row % a.period;
    if (a.positions) p = a.wide_positions ? static_cast<const int64_t*>(a.positions)[row] : static_cast<const int32_t*>(a.positions)[row];
    return p >= 0 && p < a.table_rows ? (int)p : -1;
}

// One wave for each head: any dim, any number of rotated values.
template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void qk_head_kernel(QkArgs a, int64_t block0) {
    const int lane = threadIdx.x & 63, heads = a.heads[0] + a.heads[1];
    const int64_t item = (block0 + blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
    if (item >= (int64_t)a.rows * heads) return;
    const int row = (int)(item / heads);
    int h = (int)(item % heads);
    const int which = h >= a.heads[0];
    h -= which * a.heads[0];
    const TX* x = static_cast<const TX*>(a.in[which]) + row * a.stride[which] + (int64_t)h * a.dim;
    TX* y = static_cast<TX*>(a.out[which]) + row * a.out_stride[which] + (int64_t)h * a.dim;
    const TW* w = static_cast<const TW*>(a.weight[which]);
    double sum = 0.;
    for (int i = lane; i < a.dim; i += 64) {
        const double v = to_f32(x[i]);
        sum = __builtin_fma(v, v, sum);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m);
    const double rho = rsqrt64(sum / a.dim + (double)a.eps);
    auto normed = [&](int i) { return (float)((double)to_f32(x[i]) * rho) * (w ? to_f32(w[i]) : 1.f); };
    const int half = a.rotated / 2, at = half ? table_row(a, row) : 0;
    for (int i = lane; i < half; i += 64) {
        const int i0 = a.interleaved ? 2 * i : i, i1 = a.interleaved ? 2 * i + 1 : i + half;
        const float u = normed(i0), v = normed(i1);
        const float c = at < 0 ? __builtin_nanf("") : a.cos[(int64_t)at * half + i];
        const float s = at < 0 ? __builtin_nanf("") : a.sin[(int64_t)at * half + i];
        store1(y + i0, u * c - v * s);
        store1(y + i1, v * c + u * s);
    }
    for (int i = a.rotated + lane; i < a.dim; i += 64) store1(y + i, normed(i));
}

template <typename TX, typename TW>
hipError_t launch(const QkArgs& a) {
    const int64_t items = (int64_t)a.rows * (a.heads[0] + a.heads[1]);
    return by_blocks((items + kThreads / 64 - 1) / (kThreads / 64), kThreads, [&](int64_t first, unsigned count) {
        hipLaunchKernelGGL((qk_head_kernel<TX, TW>), dim3(count), dim3(kThreads), 0, a.stream, a, first);
    });
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkArgs& a) {
    if (a.rows < 1 || a.heads[0] < 1 || a.heads[1] < 1 || a.dim < 1 || a.dim > GDR_QK_MAX_DIM || a.rotated > a.dim)
        return hipErrorInvalidValue;
    QkArgs b = a;
    b.period = a.period < 1 ? 1 : a.period;  // not used where it may be less
    if (!a.bf16) return launch<float, float>(b);
    return a.w_bf16 ? launch<bf16_t, bf16_t>(b) : launch<bf16_t, float>(b);
}

}  // namespace gdr

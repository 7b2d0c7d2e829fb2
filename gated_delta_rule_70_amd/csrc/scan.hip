// Selective scan: the recurrence with a diagonal transition that depends on the input
// (gdr_selective_scan, gdr_selective_scan_step).
#include "layer_launch.h"

#include "row_device.h"

namespace gdr {

namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(v); }

// Sixteen lanes for each channel, S state values in each: lane l has values l, l + 16, ...
template <typename TX, typename TDT, int S>
__global__ __launch_bounds__(kThreads) void scan_kernel(ScanArgs a, int tiles, int64_t block0) {
    const int64_t b = block0 + blockIdx.x;
    const int seq = (int)(b / tiles), lane = threadIdx.x & 15;
    const int d = (int)(b % tiles) * (kThreads / 16) + threadIdx.x / 16;
    if (d >= a.D) return;  // whole rows of 16 lanes
    const int N = a.N, g = d / (a.D / a.G);
    int64_t first = (int64_t)seq * a.T;
    int len = a.T;
    if (a.cu) {
        const Span s = packed_span(a.cu, seq, a.T);
        first = s.first, len = s.count;
    }
    float A[S], h[S];
    const int64_t at = ((int64_t)seq * a.D + d) * N;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int n = lane + 16 * s;
        A[s] = n < N && len > 0 ? a.A[(int64_t)d * N + n] * kLog2e : 0.f;
        h[s] = n < N && a.h0 ? a.h0[at + n] : 0.f;
    }
    const float skip = a.skip ? a.skip[d] : 0.f, bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const TX* x = static_cast<const TX*>(a.x) + first * a.x_stride + d;
    const TDT* dt = static_cast<const TDT*>(a.dt) + first * a.dt_stride + d;
    const TX* z = a.z ? static_cast<const TX*>(a.z) + first * a.z_stride + d : nullptr;
    const TX* B = static_cast<const TX*>(a.b) + first * a.b_stride + (int64_t)g * N;
    const TX* C = static_cast<const TX*>(a.c) + first * a.c_stride + (int64_t)g * N;
    TX* out = static_cast<TX*>(a.out) + first * a.out_stride + d;
    for (int t = 0; t < len; ++t) {
        const float xv = to_f32(x[t * a.x_stride]);
        float step = to_f32(dt[t * a.dt_stride]) + bias;
        if (a.softplus) step = softplus(step);
        const float in = step * xv;
        float y = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int n = lane + 16 * s;
            const float bv = n < N ? to_f32(B[t * a.b_stride + n]) : 0.f, cv = n < N ? to_f32(C[t * a.c_stride + n]) : 0.f;
            h[s] = __builtin_fmaf(__builtin_amdgcn_exp2f(step * A[s]), h[s], in * bv);
            y = __builtin_fmaf(cv, h[s], y);
        }
        y = row_sum(y);
        y = __builtin_fmaf(skip, xv, y);
        if (z) y *= silu(to_f32(z[t * a.z_stride]));
        if (lane == 0) store1(out + t * a.out_stride, y);
    }
    if (a.ht)
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (lane + 16 * s < N) a.ht[at + lane + 16 * s] = h[s];
}

template <typename TX, typename TDT>
hipError_t launch(const ScanArgs& a) {
    const int tiles = (a.D + kThreads / 16 - 1) / (kThreads / 16);
    return by_blocks((int64_t)a.B * tiles, kThreads, [&](int64_t first, unsigned count) {
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(count), dim3(kThreads), 0, a.stream, a, tiles, first); };
        if (a.N <= 16)
            go(scan_kernel<TX, TDT, 1>);
        else if (a.N <= 32)
            go(scan_kernel<TX, TDT, 2>);
        else if (a.N <= 64)
            go(scan_kernel<TX, TDT, 4>);
        else
            go(scan_kernel<TX, TDT, 8>);
    });
}

hipError_t typed(const ScanArgs& a) {
    if (a.B < 1 || a.D < 1 || a.N < 1 || a.N > GDR_SCAN_MAX_STATES || a.G < 1 || a.D % a.G) return hipErrorInvalidValue;
    if (!a.bf16) return launch<float, float>(a);
    return a.dt_bf16 ? launch<bf16_t, bf16_t>(a) : launch<bf16_t, float>(a);
}

}  // namespace

hipError_t launch_selective_scan(const ScanArgs& a) { return typed(a); }
hipError_t launch_selective_scan_step(const ScanArgs& a) { return typed(a); }

}  // namespace gdr

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

// P lanes for each head (a power of two, at least dim / 16), sixteen values in each: lane l of the
// first rotated / 16 has both halves of the pairs 8 l .. 8 l + 7, so nothing is exchanged but the sum of
// squares.  A wave has 64 / P heads of a row at once and U such groups one after the other, all loaded
// before the first is normed, and reads its part of the tables once for them.
template <typename TX, typename TW, int P, int U>
__global__ __launch_bounds__(kThreads) void qk_kernel(QkArgs a, int q_parts, int parts, int64_t block0) {
    constexpr int H = 64 / P;
    const int64_t item = (block0 + blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
    if (item >= (int64_t)a.rows * parts) return;
    const int row = (int)(item / parts), part = (int)(item % parts), which = part >= q_parts;
    const int lane = threadIdx.x % P, h0 = (part - which * q_parts) * (H * U) + (threadIdx.x & 63) / P;
    const int heads = a.heads[which], turned = a.rotated / 16;
    const bool mine = lane < a.dim / 16;
    const bool halves = !a.interleaved && lane < turned;
    const int e0 = halves ? 8 * lane : a.interleaved ? 16 * lane : a.rotated + 16 * (lane - turned);
    const int e1 = halves ? a.rotated / 2 + 8 * lane : e0 + 8;
    const TX* x = static_cast<const TX*>(a.in[which]) + row * a.stride[which];
    TX* y = static_cast<TX*>(a.out[which]) + row * a.out_stride[which];

    float u[U][8], v[U][8];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int h = h0 + i * H;
        if (mine && h < heads) {
            load8<false>(x + (int64_t)h * a.dim + e0, 8, u[i]);
            load8<false>(x + (int64_t)h * a.dim + e1, 8, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[i][j] = v[i][j] = 0.f;
        }
    }
    float w0[8], w1[8], c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w0[j] = w1[j] = c[j] = 1.f, s[j] = 0.f;
    if (mine && a.weight[which]) {
        load8<false>(static_cast<const TW*>(a.weight[which]) + e0, 8, w0);
        load8<false>(static_cast<const TW*>(a.weight[which]) + e1, 8, w1);
    }
    if (lane < turned) {
        const int at = table_row(a, row);
        if (at >= 0) {
            load8<false>(a.cos + (int64_t)at * (a.rotated / 2) + 8 * lane, 8, c);
            load8<false>(a.sin + (int64_t)at * (a.rotated / 2) + 8 * lane, 8, s);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = s[j] = __builtin_nanf("");
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int h = h0 + i * H;
        double sum = 0.;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = __builtin_fma((double)u[i][j], (double)u[i][j], sum);
            sum = __builtin_fma((double)v[i][j], (double)v[i][j], sum);
        }
        if constexpr (P > 1) sum += dpp_mov64<0xB1>(sum);   // quad_perm [1,0,3,2]
        if constexpr (P > 2) sum += dpp_mov64<0x4E>(sum);   // quad_perm [2,3,0,1]
        if constexpr (P > 4) sum += dpp_mov64<0x141>(sum);  // row_half_mirror
        if constexpr (P > 8) sum += dpp_mov64<0x140>(sum);  // row_mirror
        if constexpr (P > 16) sum += __shfl_xor(sum, 16);
        double rho64 = rsqrt64(sum / a.dim + (double)a.eps);
        float scale = 1.f;  // the factor may lie outside fp32's normal range where the values are near its ends
        if (rho64 > 0x1p100) scale = 0x1p64f, rho64 *= 0x1p-64;
        if (rho64 < 0x1p-100) scale = 0x1p-64f, rho64 *= 0x1p64;
        const float rho = (float)rho64;
        if (scale != 1.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[i][j] *= scale, v[i][j] *= scale;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = u[i][j] * rho * w0[j], v[i][j] = v[i][j] * rho * w1[j];
        if (lane < turned) {
            if (!a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = u[i][j], q = v[i][j];
                    u[i][j] = p * c[j] - q * s[j];
                    v[i][j] = q * c[j] + p * s[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float* t = j < 4 ? &u[i][2 * j] : &v[i][2 * (j - 4)];
                    const float p = t[0], q = t[1];
                    t[0] = p * c[j] - q * s[j];
                    t[1] = q * c[j] + p * s[j];
                }
            }
        }
        if (mine && h < heads) {
            store8<false>(y + (int64_t)h * a.dim + e0, 8, u[i]);
            store8<false>(y + (int64_t)h * a.dim + e1, 8, v[i]);
        }
    }
}

template <typename TX, typename TW, int P, int U>
hipError_t launch_lanes(const QkArgs& a) {
    constexpr int at_once = 64 / P * U;
    const int q_parts = (a.heads[0] + at_once - 1) / at_once, parts = q_parts + (a.heads[1] + at_once - 1) / at_once;
    const int64_t items = (int64_t)a.rows * parts;
    return by_blocks((items + kThreads / 64 - 1) / (kThreads / 64), kThreads, [&](int64_t first, unsigned count) {
        hipLaunchKernelGGL((qk_kernel<TX, TW, P, U>), dim3(count), dim3(kThreads), 0, a.stream, a, q_parts, parts, first);
    });
}

template <typename TX, typename TW, int P>
hipError_t launch_lanes(const QkArgs& a) {
    constexpr int H = 64 / P;
    return a.heads[0] > H && (int64_t)a.rows * (a.heads[0] + a.heads[1]) >= 16384 * H ? launch_lanes<TX, TW, P, 2>(a) : launch_lanes<TX, TW, P, 1>(a);
}

template <typename TX, typename TW>
hipError_t launch(const QkArgs& a) {
    if (a.dim % 16 == 0 && a.rotated % 16 == 0) {
        const int lanes = a.dim / 16;
        return lanes <= 1    ? launch_lanes<TX, TW, 1>(a)
               : lanes <= 2  ? launch_lanes<TX, TW, 2>(a)
               : lanes <= 4  ? launch_lanes<TX, TW, 4>(a)
               : lanes <= 8  ? launch_lanes<TX, TW, 8>(a)
               : lanes <= 16 ? launch_lanes<TX, TW, 16>(a)
                             : launch_lanes<TX, TW, 32>(a);
    }
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

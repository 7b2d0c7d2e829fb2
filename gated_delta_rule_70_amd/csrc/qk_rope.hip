// Root-mean-square norm of query and key heads with the rotation by position (gdr_qk_norm_rope).
//
// n = x / sqrt(mean x^2 + eps) * w, then (a, b) -> (a c - b s, b c + a s) on pairs.  Bound by memory: every head
// is read and written once, in one pass, and a row's part of the tables comes from the caches for all heads
// but the first.  4097 rows of 32 + 16 heads of 128, bf16, 22 us from one call to the next (4.6 TB/s; 28 with
// inputs from memory), 32768 rows 159 (5.1); heads of 90, in overlapping groups, 24.  The angles come from tables, so far
// positions lose nothing; squares are summed in fp64, whose range no bf16 or fp32 head leaves; everything else
// is fp32, rounded once.
#include "layer_launch.h"

#include "row_device.h"

namespace gdr {

namespace {

constexpr int kThreads = 256;

// The row of the tables that a row of q and k takes, or -1.
__device__ __forceinline__ int table_row(const QkArgs& a, int row) {
    int64_t p = row % a.period;
    if (a.positions) p = a.wide_positions ? static_cast<const int64_t*>(a.positions)[row] : static_cast<const int32_t*>(a.positions)[row];
    return p >= 0 && p < a.table_rows ? (int)p : -1;
}

// How a head's parts (the pairs that are rotated, the values that are not) go into groups of eight.
enum {
    kWhole,    // both without rest
    kOverlap,  // the last group of a part begins earlier, so that it is whole: some values are computed twice
    kPart      // a part has fewer than eight: value by value
};

// P lanes for each head (a power of two), sixteen values in each: lane l of the first `turned` has both
// halves of the pairs 8 l .. 8 l + 7, so nothing is exchanged but the sum of squares; the others have
// sixteen of the values that are not rotated.  A wave has 64 / P heads of a row (twice as many, one after the
// other, were 1 % faster at 4097 x 48 x 128 and no faster at 16384 x 40 x 64).
template <typename TX, typename TW, int P, int FORM>
__global__ __launch_bounds__(kThreads) void qk_kernel(QkArgs a, int q_parts, int parts, int64_t block0) {
    constexpr int H = 64 / P;
    constexpr bool PART = FORM == kPart;
    const int64_t item = (block0 + blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
    if (item >= (int64_t)a.rows * parts) return;
    const int row = (int)(item / parts), part = (int)(item % parts), which = part >= q_parts;
    const int lane = threadIdx.x % P, h = (part - which * q_parts) * H + (threadIdx.x & 63) / P;
    const int heads = a.heads[which], turned = (a.rotated + 15) / 16, rest = lane - turned;
    const bool halves = !a.interleaved && rest < 0;
    int e0 = halves ? 8 * lane : rest < 0 ? 16 * lane : a.rotated + 16 * rest;
    int e1 = halves ? a.rotated / 2 + 8 * lane : e0 + 8;
    const int until = halves ? a.rotated / 2 : rest < 0 ? a.rotated : a.dim;  // the values of this part
    const int n0 = until - e0, n1 = halves ? n0 : until - e1;
    const bool mine = n0 > 0;
    int twice0 = 0, twice1 = 0;  // values at the beginning that another group has, too
    if constexpr (FORM == kOverlap) {
        twice0 = n0 < 8 ? 8 - n0 : 0, twice1 = n1 < 8 ? 8 - n1 : 0;
        e0 -= twice0, e1 -= twice1;
    }
    const TX* x = static_cast<const TX*>(a.in[which]) + row * a.stride[which];
    TX* y = static_cast<TX*>(a.out[which]) + row * a.out_stride[which];

    float u[8], v[8];
    if (mine && h < heads) {
        load8<PART>(x + (int64_t)h * a.dim + e0, n0, u);
        load8<PART>(x + (int64_t)h * a.dim + e1, n1, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = v[j] = 0.f;
    }
    float w0[8], w1[8], c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w0[j] = w1[j] = c[j] = 1.f, s[j] = 0.f;
    if (mine && a.weight[which]) {
        load8<PART>(static_cast<const TW*>(a.weight[which]) + e0, n0, w0);
        load8<PART>(static_cast<const TW*>(a.weight[which]) + e1, n1, w1);
    }
    if (rest < 0) {
        const int at = table_row(a, row);
        const int64_t from = (int64_t)at * (a.rotated / 2);
        if (at < 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = s[j] = __builtin_nanf("");
        } else if (FORM == kOverlap && a.interleaved) {  // four pairs each
            __builtin_memcpy(c, a.cos + from + e0 / 2, 16);
            __builtin_memcpy(c + 4, a.cos + from + e1 / 2, 16);
            __builtin_memcpy(s, a.sin + from + e0 / 2, 16);
            __builtin_memcpy(s + 4, a.sin + from + e1 / 2, 16);
        } else {
            const int first = halves ? e0 : e0 / 2;
            load8<PART>(a.cos + from + first, a.rotated / 2 - first, c);
            load8<PART>(a.sin + from + first, a.rotated / 2 - first, s);
        }
    }
    double sum = 0.;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float p = FORM == kOverlap && j < twice0 ? 0.f : u[j], q = FORM == kOverlap && j < twice1 ? 0.f : v[j];
        sum = __builtin_fma((double)p, (double)p, sum);
        sum = __builtin_fma((double)q, (double)q, sum);
    }
    if constexpr (P > 1) sum += dpp_mov64<0xB1>(sum);   // quad_perm [1,0,3,2]
    if constexpr (P > 2) sum += dpp_mov64<0x4E>(sum);   // quad_perm [2,3,0,1]
    if constexpr (P > 4) sum += dpp_mov64<0x141>(sum);  // row_half_mirror
    if constexpr (P > 8) sum += dpp_mov64<0x140>(sum);  // row_mirror
    if constexpr (P > 16) sum += __shfl_xor(sum, 16);
    if constexpr (P > 32) sum += __shfl_xor(sum, 32);
    double rho64 = rsqrt64(sum / a.dim + (double)a.eps);
    float scale = 1.f;  // the factor may lie outside fp32's normal range where the values are near its ends
    if (rho64 > 0x1p100) scale = 0x1p64f, rho64 *= 0x1p-64;
    if (rho64 < 0x1p-100) scale = 0x1p-64f, rho64 *= 0x1p64;
    const float rho = (float)rho64;
    if (scale != 1.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] *= scale, v[j] *= scale;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = u[j] * rho * w0[j], v[j] = v[j] * rho * w1[j];
    if (rest < 0) {
        if (!a.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = u[j], q = v[j];
                u[j] = p * c[j] - q * s[j];
                v[j] = q * c[j] + p * s[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float* t = j < 4 ? &u[2 * j] : &v[2 * (j - 4)];
                const float p = t[0], q = t[1];
                t[0] = p * c[j] - q * s[j];
                t[1] = q * c[j] + p * s[j];
            }
        }
    }
    if (mine && h < heads) {
        store8<PART>(y + (int64_t)h * a.dim + e0, n0, u);
        store8<PART>(y + (int64_t)h * a.dim + e1, n1, v);
    }
}

template <typename TX, typename TW, int P, int FORM>
hipError_t launch_lanes(const QkArgs& a) {
    constexpr int at_once = 64 / P;
    const int q_parts = (a.heads[0] + at_once - 1) / at_once, parts = q_parts + (a.heads[1] + at_once - 1) / at_once;
    const int64_t items = (int64_t)a.rows * parts;
    return by_blocks((items + kThreads / 64 - 1) / (kThreads / 64), kThreads, [&](int64_t first, unsigned count) {
        hipLaunchKernelGGL((qk_kernel<TX, TW, P, FORM>), dim3(count), dim3(kThreads), 0, a.stream, a, q_parts, parts, first);
    });
}

template <typename TX, typename TW, int P>
hipError_t launch_lanes(const QkArgs& a) {
    const int pairs = a.interleaved ? a.rotated : a.rotated / 2, rest = a.dim - a.rotated;
    if ((pairs > 0 && pairs < 8) || (rest > 0 && rest < 8)) return launch_lanes<TX, TW, P, kPart>(a);
    if (a.rotated % 16 || a.dim % 16) return launch_lanes<TX, TW, P, kOverlap>(a);
    if constexpr (P == 64)
        return hipErrorInvalidValue;  // more than 32 lanes: never without rest
    else
        return launch_lanes<TX, TW, P, kWhole>(a);
}

template <typename TX, typename TW>
hipError_t launch(const QkArgs& a) {
    const int lanes = (a.rotated + 15) / 16 + (a.dim - a.rotated + 15) / 16;
    return lanes <= 1    ? launch_lanes<TX, TW, 1>(a)
           : lanes <= 2  ? launch_lanes<TX, TW, 2>(a)
           : lanes <= 4  ? launch_lanes<TX, TW, 4>(a)
           : lanes <= 8  ? launch_lanes<TX, TW, 8>(a)
           : lanes <= 16 ? launch_lanes<TX, TW, 16>(a)
           : lanes <= 32 ? launch_lanes<TX, TW, 32>(a)
                         : launch_lanes<TX, TW, 64>(a);
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

// Device-side helpers of the kernels that work on rows of values: loads and stores of eight
// values at any alignment, sums over the lanes that share a head, exponentials.
#pragma once

#include "gdr_device.h"

namespace gdr {

// Values 0 .. 7 at p as fp32, zeros from n on.  Vector loads at any alignment of the elements: the
// hardware takes them unaligned, so only a row's last group of fewer than 8 (PART: there may be
// one) goes value by value.
template <bool PART>
__device__ __forceinline__ void load8(const bf16_t* p, int n, float (&v)[8]) {
    if (!PART || n >= 8) {
        u32x4 u;
        __builtin_memcpy(&u, p, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? to_f32(p[j]) : 0.f;
    }
}
template <bool PART>
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
    if (!PART || n >= 8) {
        __builtin_memcpy(v, p, 32);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.f;
    }
}
__device__ __forceinline__ float round_to(float x, const float*) { return x; }
__device__ __forceinline__ float round_to(float x, const bf16_t*) {
    return static_cast<float>(static_cast<__bf16>(x));
}
// x as it is stored, in the type of what p points to.
__device__ __forceinline__ float rounded(float x, const float*) { return x; }
__device__ __forceinline__ bf16_t rounded(float x, const bf16_t*) {
    return bf16_t{__builtin_bit_cast(uint16_t, static_cast<__bf16>(x))};
}
template <bool PART>
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
    if (!PART || n >= 8) {
        __builtin_memcpy(p, v, 32);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = v[j];
    }
}
template <bool PART>
__device__ __forceinline__ void store8(bf16_t* p, int n, const float (&v)[8]) {
    const u32x2 a = bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]}), b = bf16x4_bits(f32x4{v[4], v[5], v[6], v[7]});
    const u32x4 u = {a[0], a[1], b[0], b[1]};
    if (!PART || n >= 8) {
        __builtin_memcpy(p, &u, 16);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j].bits = (uint16_t)(u[j / 2] >> (j % 2 * 16));
    }
}

// Eight values as loaded, turned to fp32 where they are used, so that the load stays in flight.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    f32x4 v[2];
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[i / 4][i % 4];
    }
};
template <>
struct Raw8<bf16_t> {
    u32x4 v;
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    }
};
template <bool PART, typename T>
__device__ __forceinline__ Raw8<T> load8_raw(const T* p, int n) {
    Raw8<T> r{};
    if (!PART || n >= 8) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
        T t[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) t[i] = p[i];
        __builtin_memcpy(&r, t, sizeof(r));
    }
    return r;
}

// Sum over the V / 8 neighbouring lanes (4, 8 or 16) that hold a head's V values, in all of them.
template <int CTRL>
__device__ __forceinline__ double dpp_mov64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_head(double x, int V) {
    x += dpp_mov64<0xB1>(x);               // quad_perm [1,0,3,2]
    x += dpp_mov64<0x4E>(x);               // quad_perm [2,3,0,1]
    if (V > 32) x += dpp_mov64<0x141>(x);  // row_half_mirror: the other quad of 8 lanes
    if (V > 64) x += dpp_mov64<0x140>(x);  // row_mirror: the other half of 16 lanes
    return x;
}

// 1 / sqrt(m) in fp64: the hardware's estimate and one Newton step.  Zero for m = 0.
__device__ __forceinline__ double rsqrt64(double m) {
    const double r = __builtin_amdgcn_rsq(m);
    const double e = __builtin_fma(-m * r, r, 1.0);
    return m == 0. ? 0. : __builtin_fma(r * 0.5, e, r);
}

// exp(-z) to about 1 ulp: the product with log2(e) is taken in two parts, so that the error of
// the exponent does not grow with |z|.  Beyond |z| = 200 the result stays infinity or zero.
__device__ __forceinline__ float exp_neg(float z) {
    z = __builtin_amdgcn_fmed3f(z, -200.f, 200.f);
    constexpr float kL = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;  // log2(e), high and low
    const float p = -z * kL;
    const float e = __builtin_fmaf(-z, kL, -p) + -z * kLo;
    return __builtin_amdgcn_exp2f(p) * __builtin_fmaf(e, 0.6931471805599453f, 1.f);
}

// z / (1 + exp(-z))
__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.f + exp_neg(z)); }

constexpr float kLog2e = 1.44269504088896341f;

// silu(z) for an fp32 output, and for a bf16 one, where the exponent's error of |z| 2^-24 does not show.
__device__ __forceinline__ float silu_for(float z, const float*) { return silu(z); }
__device__ __forceinline__ float silu_for(float z, const bf16_t*) {
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|), to a few ulp of the result at any v: far
// below zero it is exp(v), for which 1 + exp(v) has no bits.  log1p(e) = 2 artanh(s) with
// s = e / (2 + e) <= 1/3; artanh(s) / s is a polynomial in s^2 <= 1/9 through its Chebyshev nodes,
// within 2^-26 of it.
__device__ __forceinline__ float softplus(float v) {
    const float e = exp_neg(fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float p = 0.1408732831478119f;
    p = __builtin_fmaf(p, q, 0.1398070901632309f);
    p = __builtin_fmaf(p, q, 0.20012426376342773f);
    p = __builtin_fmaf(p, q, 0.3333315849304199f);
    p = __builtin_fmaf(p, q, 1.f);
    const float r = __builtin_fmaf(2.f * s, p, fmaxf(v, 0.f));
    return v != v ? v : r;
}

constexpr int kXcds = 8;

// Work item of block b of n, so that each XCD (block b is on XCD b % 8) has a contiguous range: what
// neighbouring items share is then in its L2.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t n) {
    const int64_t q = n / kXcds, r = n % kXcds, x = b % kXcds;
    return x * q + (x < r ? x : r) + b / kXcds;
}

// A sequence's rows in a packed batch of T rows: clamped, so that no entry leads outside.
struct Span {
    int first, count;
};
__device__ __forceinline__ Span packed_span(const int32_t* cu, int i, int T) {
    const int a = min(max(cu[i], 0), T);
    return Span{a, min(max(cu[i + 1], a), T) - a};
}

}  // namespace gdr

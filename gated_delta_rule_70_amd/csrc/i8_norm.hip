// Norms that give int8 codes and a scale for each row: the residual addition with a
// root-mean-square norm, and the norm per value head times silu(gate).
//
// One pass over memory.  With s the row to be normed, t = s * weight, A = max |t| and
// rho = (mean s^2 + eps)^(-1/2), the code of the normed value t * rho at scale A * rho / 127 is
// rint(127 t / A): rho cancels.  So the sum of squares and the maximum are reduced together,
// the row stays in registers in between, and codes are stored after one reduction.
#include "i8_launch.h"

#include <type_traits>

#include "gdr_device.h"

namespace gdr {

namespace {

constexpr float kFltMax = 3.402823466e38f;

// Eight consecutive values as fp32.  WIDE: the address takes 16-byte loads.
template <bool WIDE>
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
    if constexpr (WIDE) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f32(p[j]);
    }
}
template <bool WIDE>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    if constexpr (WIDE) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p[j];
    }
}
__device__ __forceinline__ float round_to(float x, const float*) { return x; }
__device__ __forceinline__ float round_to(float x, const bf16_t*) {
    return static_cast<float>(static_cast<__bf16>(x));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(bf16_t* p, float x) { *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(x); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
    const u32x2 a = bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]}), b = bf16x4_bits(f32x4{v[4], v[5], v[6], v[7]});
    *reinterpret_cast<u32x4*>(p) = u32x4{a[0], a[1], b[0], b[1]};
}
__device__ __forceinline__ u32x2 pack8(const int (&c)[8]) {
    u32x2 r;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        r[j] = (c[4 * j] & 0xFF) | (c[4 * j + 1] & 0xFF) << 8 | (c[4 * j + 2] & 0xFF) << 16 | (uint32_t)c[4 * j + 3] << 24;
    return r;
}

// Sum and maximum of TPR consecutive threads (64, or the whole workgroup), in all of them.
template <int TPR, typename T>
__device__ __forceinline__ void reduce_row(double& sum, T& top, int& bad) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        sum += __shfl_xor(sum, m);
        const T o = __shfl_xor(top, m);
        top = o > top ? o : top;
    }
    bad = __any(bad);
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        __shared__ double s_sum[NW];
        __shared__ T s_top[NW];
        __shared__ int s_bad[NW];
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) s_sum[wave] = sum, s_top[wave] = top, s_bad[wave] = bad;
        __syncthreads();
        sum = s_sum[0], top = s_top[0], bad = s_bad[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) {
            sum += s_sum[i];
            top = s_top[i] > top ? s_top[i] : top;
            bad |= s_bad[i];
        }
    }
}

// Residual addition, norm and codes.  TPR threads for each row, NV groups of 8 values in each
// thread: WIDE groups are 8 consecutive values, otherwise values TPR apart (so that single
// loads of neighbouring threads are neighbours).
//
// T holds t: fp32 where s and weight are bf16 (a product of two 8-bit significands is exact),
// fp64 otherwise (exact again), so A is exact too.  127 t / A is taken in fp32 first: its error
// is below 4 * 2^-24 relative, 2^-15 absolute; within 2^-14 of a border between codes (one value
// in 8000) it is taken again in fp64.
template <typename TX, typename TW, typename T, int TPR, int NV, bool WIDE>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_rmsnorm_kernel(NormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const int tid = TPR < 256 ? threadIdx.x % TPR : threadIdx.x;
    const int row = blockIdx.x * RPB + (TPR < 256 ? threadIdx.x / TPR : 0);
    if (TPR < 256 && row >= a.rows) return;  // whole waves: no barrier is used then
    const int D = a.cols;
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride;
    const TX* r = a.r ? static_cast<const TX*>(a.r) + row * a.r_stride : nullptr;
    TX* out = a.out ? static_cast<TX*>(a.out) + row * a.out_stride : nullptr;
    const TW* w = static_cast<const TW*>(a.w);
    int8_t* q = a.q + (int64_t)row * D;

    T t[NV][8];
    double sum = 0.;
    T top = T(0);
    int bad = 0;
    auto at = [&](int i, int j) { return WIDE ? (i * TPR + tid) * 8 + j : (i * 8 + j) * TPR + tid; };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s[8], wv[8];
        if constexpr (WIDE) {
            if (at(i, 0) < D) {
                load8<true>(x + at(i, 0), s);
                load8<true>(w + at(i, 0), wv);
                if (r) {
                    float rv[8];
                    load8<true>(r + at(i, 0), rv);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] = round_to(s[j] + rv[j], x);
                }
                if (out) store8(out + at(i, 0), s);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = wv[j] = 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = at(i, j);
                s[j] = wv[j] = 0.f;
                if (e < D) {
                    s[j] = to_f32(x[e]);
                    wv[j] = to_f32(w[e]);
                    if (r) s[j] = round_to(s[j] + to_f32(r[e]), x);
                    if (out) store1(out + e, s[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = __builtin_fma((double)s[j], (double)s[j], sum);
            t[i][j] = (T)s[j] * (T)wv[j];
            const T m = t[i][j] < T(0) ? -t[i][j] : t[i][j];
            bad |= !(m <= T(kFltMax));
            top = m > top ? m : top;
        }
    }
    reduce_row<TPR>(sum, top, bad);

    const double rho = 1.0 / sqrt(sum / D + (double)a.eps);
    if (tid == 0) {
        double sc = (double)top * rho / 127.0;
        if (top == T(0)) sc = 0.;  // also with eps = 0, where rho is infinite
        a.scale[row] = bad ? __builtin_nanf("") : (float)sc;
    }
    const bool zero = bad || top == T(0);
    // below 2^-100 the quotient's fp32 form would overflow: every code is taken in fp64
    const bool tiny = top < T(0x1p-100f);
    const float inv = zero || tiny ? 0.f : 127.f / (float)top;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int c[8];
        float worst = tiny ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = (float)t[i][j] * inv, n = __builtin_rintf(v);
            c[j] = (int)n;
            worst = fmaxf(worst, fabsf(v - n));
        }
        if (worst > 0.5f - 0x1p-14f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = zero ? 0 : (int)rint((double)t[i][j] * 127.0 / (double)top);
        }
        if (zero) {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = 0;
        }
        if constexpr (WIDE) {
            if (at(i, 0) < D) *reinterpret_cast<u32x2*>(q + at(i, 0)) = pack8(c);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(i, j) < D) q[at(i, j)] = (int8_t)c[j];
        }
    }
}

// exp(-z) to about 1 ulp: the product with log2(e) is taken in two parts, so that the error of
// the exponent does not grow with |z|.  Beyond |z| = 200 the result stays infinity or zero.
__device__ __forceinline__ float exp_neg(float z) {
    z = fminf(fmaxf(z, -200.f), 200.f);
    constexpr float kL = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;  // log2(e), high and low
    const float p = -z * kL;
    const float e = __builtin_fmaf(-z, kL, -p) + -z * kLo;
    return __builtin_amdgcn_exp2f(p) * __builtin_fmaf(e, 0.6931471805599453f, 1.f);
}

// Norm per value head (V values, V/8 neighbouring threads), times weight and silu(gate), and
// codes over the whole token.
template <typename TO, typename TG, typename TW, int TPR, int NV, bool WIDE>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void gated_rmsnorm_kernel(NormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const int tid = TPR < 256 ? threadIdx.x % TPR : threadIdx.x;
    const int row = blockIdx.x * RPB + (TPR < 256 ? threadIdx.x / TPR : 0);
    if (TPR < 256 && row >= a.rows) return;
    const int V = a.cols, D = a.heads * V;
    const TO* o = static_cast<const TO*>(a.x) + row * a.x_stride;
    const TG* z = static_cast<const TG*>(a.r) + row * a.r_stride;
    const TW* w = static_cast<const TW*>(a.w);
    int8_t* q = a.q + (int64_t)row * D;

    float n[NV][8];
    uint32_t top = 0;  // |n| as ordered bits: NaN above infinity above every number
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + tid) * 8;
        float zv[8], wv[8];
        if (e < D) {
            load8<WIDE>(o + e, n[i]);
            load8<WIDE>(z + e, zv);
            load8<WIDE>(w + e % V, wv);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) n[i][j] = zv[j] = wv[j] = 0.f;
        }
        double ss = 0.;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)n[i][j], (double)n[i][j], ss);
        for (int m = V / 16; m >= 1; m >>= 1) ss += __shfl_xor(ss, m);
        const float rho = (float)(1.0 / sqrt(ss / V + (double)a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // a zero head stays zero also where eps = 0 makes rho infinite
            const float x = n[i][j] == 0.f ? 0.f : n[i][j] * rho;
            n[i][j] = x * wv[j] * (zv[j] / (1.f + exp_neg(zv[j])));
            const uint32_t b = __float_as_uint(n[i][j]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
    }
    double none = 0.;
    int bad = top >= 0x7F800000u;
    reduce_row<TPR>(none, top, bad);
    const float A = __uint_as_float(top);
    const bool zero = bad || top == 0;
    if (tid == 0) a.scale[row] = bad ? __builtin_nanf("") : A / 127.f;
    // a power of two that keeps 127 / A finite
    const float up = A < 0x1p-100f ? 0x1p100f : 1.f;
    const float inv = zero ? 0.f : 127.f / (A * up);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + tid) * 8;
        int c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = zero ? 0 : (int)__builtin_rintf(n[i][j] * up * inv);
        if (e < D) {
            if constexpr (WIDE)
                *reinterpret_cast<u32x2*>(q + e) = pack8(c);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) q[e + j] = (int8_t)c[j];
        }
    }
}

bool wide(const void* p, int64_t stride, int rows, int elt) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows == 1 || stride * elt % 16 == 0));
}

template <int TPR>
dim3 grid_of(int rows) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    return dim3((unsigned)((rows + (int64_t)RPB - 1) / RPB));
}

template <typename TX, typename TW, typename T, bool WIDE>
void add_rmsnorm_sized(const NormArgs& a) {
    auto go = [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        hipLaunchKernelGGL((add_rmsnorm_kernel<TX, TW, T, TPR, NV, WIDE>), grid_of<TPR>(a.rows),
                           dim3(TPR < 256 ? 256 : TPR), 0, a.stream, a);
    };
    using std::integral_constant;
    if (a.cols <= 512)
        go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (a.cols <= 2048)
        go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    else if (a.cols <= 4096)
        go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (a.cols <= 8192)
        go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    else
        go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <typename TX, typename TW, typename T>
void add_rmsnorm_typed(const NormArgs& a) {
    const bool v = a.cols % 8 == 0 && wide(a.x, a.x_stride, a.rows, sizeof(TX)) &&
                   wide(a.r, a.r_stride, a.rows, sizeof(TX)) && wide(a.out, a.out_stride, a.rows, sizeof(TX)) &&
                   wide(a.w, 0, 1, sizeof(TW)) && wide(a.q, a.cols, 1, 1);
    v ? add_rmsnorm_sized<TX, TW, T, true>(a) : add_rmsnorm_sized<TX, TW, T, false>(a);
}

template <typename TO, typename TG, typename TW, bool WIDE>
void gated_sized(const NormArgs& a) {
    auto go = [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        hipLaunchKernelGGL((gated_rmsnorm_kernel<TO, TG, TW, TPR, NV, WIDE>), grid_of<TPR>(a.rows),
                           dim3(TPR < 256 ? 256 : TPR), 0, a.stream, a);
    };
    using std::integral_constant;
    const int D = a.heads * a.cols;
    if (D <= 512)
        go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (D <= 4096)
        go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (D <= 8192)
        go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    else
        go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <typename TO, typename TG, typename TW>
void gated_typed(const NormArgs& a) {
    const bool v = wide(a.x, a.x_stride, a.rows, sizeof(TO)) && wide(a.r, a.r_stride, a.rows, sizeof(TG)) &&
                   wide(a.w, 0, 1, sizeof(TW)) && wide(a.q, a.heads * a.cols, 1, 1);
    v ? gated_sized<TO, TG, TW, true>(a) : gated_sized<TO, TG, TW, false>(a);
}

}  // namespace

hipError_t launch_add_rmsnorm_i8(const NormArgs& a) {
    if (a.rows < 1 || a.cols < 1 || a.cols > GDR_NORM_MAX_COLS) return hipErrorInvalidValue;
    if (!a.x_bf16)
        add_rmsnorm_typed<float, float, double>(a);
    else if (a.w_bf16)
        add_rmsnorm_typed<bf16_t, bf16_t, float>(a);
    else
        add_rmsnorm_typed<bf16_t, float, double>(a);
    return hipGetLastError();
}

hipError_t launch_gated_rmsnorm_i8(const NormArgs& a) {
    if (a.rows < 1 || a.heads * a.cols > GDR_NORM_MAX_COLS || a.cols % 32 != 0 || a.cols > 128)
        return hipErrorInvalidValue;
    auto w = [&](auto o, auto g) {
        a.w_bf16 ? gated_typed<decltype(o), decltype(g), bf16_t>(a) : gated_typed<decltype(o), decltype(g), float>(a);
    };
    auto g = [&](auto o) { a.gate_bf16 ? w(o, bf16_t{}) : w(o, float{}); };
    a.x_bf16 ? g(bf16_t{}) : g(float{});
    return hipGetLastError();
}

}  // namespace gdr

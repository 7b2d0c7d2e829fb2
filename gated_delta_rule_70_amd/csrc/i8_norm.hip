// Norms that give int8 codes and a scale for each row: the residual addition with a
// root-mean-square norm, and the norm per value head times silu(gate).
//
// One pass over memory.  With s the row to be normed, t = s * weight, A = max |t| and
// rho = (mean s^2 + eps)^(-1/2), the code of the normed value t * rho at scale A * rho / 127 is
// rint(127 t / A): rho cancels.  So the sum of squares and the maximum are reduced together,
// the row stays in registers in between, and codes are stored after one reduction.  Bound by
// memory: 32768 x 4096 bf16 with residual 163 us from one call to the next, 5.8 TB/s (156 in a
// kernel trace; a copy of 1 GiB reaches 5.1, and part of what is read here is still in the last-level
// cache); 4097 tokens of 32 x 128 bf16 through the gated norm 20.0 us with inputs from memory, 4.2
// TB/s (19.9 in a trace, 17.1 with inputs in the cache), where the exponentials cost about as much
// time as the memory.
#include "i8_launch.h"

#include <type_traits>

#include "gdr_device.h"

namespace gdr {

namespace {

constexpr float kFltMax = 3.402823466e38f;

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

// Rounding to whole numbers, ties to even, by one addition: x + kRound (|x| < 2^22) has the whole
// number's low bits at its end.
constexpr float kRound = 12582912.f;  // 1.5 * 2^23
// The low bytes of eight such sums, or zeros.
__device__ __forceinline__ u32x2 pack8(const float (&y)[8], bool zero) {
    u32x2 r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t a = __builtin_amdgcn_perm(__float_as_uint(y[4 * j + 1]), __float_as_uint(y[4 * j]), 0x0C0C0400);
        const uint32_t b = __builtin_amdgcn_perm(__float_as_uint(y[4 * j + 3]), __float_as_uint(y[4 * j + 2]), 0x04000C0C);
        r[j] = zero ? 0u : a | b;
    }
    return r;
}
template <bool PART>
__device__ __forceinline__ void store_codes(int8_t* q, int n, u32x2 c) {
    if (!PART || n >= 8) {
        __builtin_memcpy(q, &c, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) q[j] = (int8_t)(c[j / 4] >> (j % 4 * 8));
    }
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

// Scale and codes of a row whose products all lie below 2^-100, with t in fp64: s is read again, from
// where this thread has just written it or from what it was made of.  Such rows are rare, so t is
// computed twice instead of being held in registers that every row would have to do without.
template <typename TX, typename TW, int TPR, bool PART>
__device__ __forceinline__ void norm_small_row(const TX* x, const TX* r, const TX* out, const TW* w, int8_t* q, float* scale,
                                               int D, int tid, double sum, float eps) {
    auto products = [&](int e, double (&t)[8]) {
        float s[8], wv[8];
        load8<PART>(out ? out + e : x + e, D - e, s);
        load8<PART>(w + e, D - e, wv);
        if (r && !out) {
            float rv[8];
            load8<PART>(r + e, D - e, rv);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = round_to(s[j] + rv[j], x);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = (double)s[j] * (double)wv[j];
    };
    double top = 0., none = 0.;
    int bad = 0;
#pragma unroll 1
    for (int e = tid * 8; e < D; e += TPR * 8) {
        double t[8];
        products(e, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmax(top, fabs(t[j]));
    }
    reduce_row<TPR>(none, top, bad);
    if (tid == 0) *scale = top == 0. ? 0.f : (float)(top * (1.0 / sqrt(sum / D + (double)eps)) / 127.0);
#pragma unroll 1
    for (int e = tid * 8; e < D; e += TPR * 8) {
        double t[8];
        products(e, t);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (top == 0. ? 0.f : (float)rint(t[j] * 127.0 / top)) + kRound;
        store_codes<PART>(q + e, D - e, pack8(y, false));
    }
}

// Residual addition, norm and codes.  TPR threads for each row, NV groups of 8 consecutive values
// in each thread.
//
// T holds t: fp32 where s and weight are bf16 (a product of two 8-bit significands is exact down
// to 2^-134; a smaller one is no longer, which matters only in rows of nothing above 2^-100: those
// are done again, see above), fp64 otherwise (exact again), so A is exact too.  127 t / A is taken in fp32 first: its error
// is below 4 * 2^-24 relative, 2^-15 absolute; within 2^-14 of a border between codes (one value
// in 8000) it is taken again in fp64.
template <typename TX, typename TW, typename T, int TPR, int NV, bool PART>
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
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + tid) * 8, n = D - e;
        float s[8] = {}, wv[8] = {};
        if (n > 0) {
            load8<PART>(x + e, n, s);
            load8<PART>(w + e, n, wv);
            if (r) {
                float rv[8];
                load8<PART>(r + e, n, rv);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = round_to(s[j] + rv[j], x);
            }
            if (out) store8<PART>(out + e, n, s);
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
    if constexpr (std::is_same_v<T, float>) {
        if (__builtin_expect(top < 0x1p-100f && sum > 0. && !bad, 0)) {  // the whole row alike
            norm_small_row<TX, TW, TPR, PART>(x, r, out, w, q, a.scale + row, D, tid, sum, a.eps);
            return;
        }
    }

    if (tid == 0) {
        const double rho = 1.0 / sqrt(sum / D + (double)a.eps);
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
        float y[8];
        float worst = tiny ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = __builtin_fmaf((float)t[i][j], inv, kRound);
            worst = fmaxf(worst, fabsf(__builtin_fmaf((float)t[i][j], inv, kRound - y[j])));
        }
        if (worst > 0.5f - 0x1p-14f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (float)rint((double)t[i][j] * 127.0 / (double)top) + kRound;
        }
        const int e = (i * TPR + tid) * 8;
        if (e < D) store_codes<PART>(q + e, D - e, pack8(y, zero));
    }
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

// Norm per value head (V values, V/8 neighbouring threads), times weight and silu(gate), and
// codes over the whole token.
template <typename TO, typename TG, typename TW, int TPR, int NV>
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

    const double per_v = V == 32 ? 1. / 32 : V == 64 ? 1. / 64 : 1. / 128;
    float n[NV][8];
    uint32_t top = 0;  // |n| as ordered bits: NaN above infinity above every number
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + tid) * 8;
        float zv[8], wv[8];
        if (e < D) {  // D is a multiple of 8
            load8<false>(o + e, 8, n[i]);
            load8<false>(z + e, 8, zv);
            load8<false>(w + (e & (V - 1)), 8, wv);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) n[i][j] = zv[j] = wv[j] = 0.f;
        }
        double ss = 0.;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)n[i][j], (double)n[i][j], ss);
        ss = sum_head(ss, V);
        double rho64 = rsqrt64(__builtin_fma(ss, per_v, (double)a.eps));
        if (rho64 > 0x1p126) {  // eps = 0 and a head of values below fp32's normal ones
            rho64 *= 0x1p-64;
#pragma unroll
            for (int j = 0; j < 8; ++j) n[i][j] *= 0x1p64f;
        }
        const float rho = (float)rho64;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float silu = zv[j] * __builtin_amdgcn_rcpf(1.f + exp_neg(zv[j]));
            n[i][j] = n[i][j] * rho * (wv[j] * silu);
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
    if (A < 0x1p-100f) {  // a power of two that keeps 127 / A finite
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) n[i][j] *= 0x1p100f;
    }
    const float inv = zero ? 0.f : 127.f / (A < 0x1p-100f ? A * 0x1p100f : A);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + tid) * 8;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(n[i][j], inv, kRound);
        if (e < D) store_codes<false>(q + e, 8, pack8(y, zero));
    }
}

template <int TPR>
dim3 grid_of(int rows) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    return dim3((unsigned)((rows + (int64_t)RPB - 1) / RPB));
}

// Threads for a row and groups for a thread: as many threads as the row fills with one or two groups
// each, since a row is read and written once and what counts is loads in flight; groups beyond a
// row's end cost time too.  A row of up to 1024 values by one wave (no barrier) pays once there are
// rows enough to fill the chip with them.  us from one call to the next, three sets of inputs in turn /
// inputs from memory; threads x groups, bf16 with residual:
//    8192 x  1024    64x2 15.7 / 19.0    64x4 16.5 / 20.2    256x1 15.9 / 19.1
//   16384 x  2048    64x4 56.6 / 57.5   256x1 43.7 / 44.9    256x2 47.3 / 47.7
//    4097 x  4096   256x2 26.6 / 26.9   512x1 25.9 / 26.1     64x8 45.5 / 45.9
//    8192 x  8192   256x4 90.3 / 92.2   512x2 84.0 / 84.4   1024x1 90.3 / 92.8
//    4096 x 16384  1024x2 86.8 / 88.3  1024x4 132 / 133
// and in the gated norm, bf16:
//    4097 x  32 x 128   512x1 17.1 / 20.0   256x2 17.5 / 20.4  1024x1 27.6 / 28.6
//    8000 x  48 x 128   512x2 56.4 / 59.6  1024x1 58.5 / 60.5
//    4097 x  64 x 128   512x2 58.0 / 58.9  1024x1 54.9 / 55.9   (fp32)
//    4097 x 128 x 128  1024x2 83.6 / 85.3  1024x4 129 / 129
template <typename TX, typename TW, typename T>
void add_rmsnorm_typed(const NormArgs& a) {
    auto go = [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const dim3 threads(TPR < 256 ? 256 : TPR);
        if (a.cols % 8 == 0)
            hipLaunchKernelGGL((add_rmsnorm_kernel<TX, TW, T, TPR, NV, false>), grid_of<TPR>(a.rows), threads, 0, a.stream, a);
        else
            hipLaunchKernelGGL((add_rmsnorm_kernel<TX, TW, T, TPR, NV, true>), grid_of<TPR>(a.rows), threads, 0, a.stream, a);
    };
    using std::integral_constant;
    if (a.cols <= 512)
        go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (a.cols <= 1024 && a.rows > 4096)
        go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (a.cols <= 2048)
        go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (a.cols <= 4096)
        go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (a.cols <= 8192)
        go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else if (a.cols <= 16384)
        go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    else
        go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <typename TO, typename TG, typename TW>
void gated_typed(const NormArgs& a) {
    auto go = [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        hipLaunchKernelGGL((gated_rmsnorm_kernel<TO, TG, TW, TPR, NV>), grid_of<TPR>(a.rows),
                           dim3(TPR < 256 ? 256 : TPR), 0, a.stream, a);
    };
    using std::integral_constant;
    const int D = a.heads * a.cols;
    if (D <= 512)
        go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (D <= 1024 && a.rows > 2048)
        go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (D <= 2048)
        go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (D <= 4096)
        go(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    else if (D <= 8192 && a.x_bf16)
        go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else if (D <= 8192)
        go(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
    else if (D <= 16384)
        go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    else
        go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

}  // namespace

// A launch has fewer than 2^32 threads: rows go in slices of 2^20, at most 1024 threads each.
template <typename F>
static hipError_t by_slices(const NormArgs& all, int64_t q_cols, F launch) {
    constexpr int kSlice = 1 << 20;
    const int64_t ex = all.x_bf16 ? 2 : 4, er = all.heads ? (all.gate_bf16 ? 2 : 4) : ex;
    for (int r0 = 0; r0 < all.rows; r0 += kSlice) {
        NormArgs a = all;
        a.rows = all.rows - r0 < kSlice ? all.rows - r0 : kSlice;
        a.x = static_cast<const char*>(all.x) + r0 * all.x_stride * ex;
        if (all.r) a.r = static_cast<const char*>(all.r) + r0 * all.r_stride * er;
        if (all.out) a.out = static_cast<char*>(all.out) + r0 * all.out_stride * ex;
        a.q += r0 * q_cols;
        a.scale += r0;
        launch(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_add_rmsnorm_i8(const NormArgs& all) {
    if (all.rows < 1 || all.rows > GDR_I8_MAX_ROWS || all.cols < 1 || all.cols > GDR_NORM_MAX_COLS)
        return hipErrorInvalidValue;
    return by_slices(all, all.cols, [](const NormArgs& a) {
        if (!a.x_bf16)
            add_rmsnorm_typed<float, float, double>(a);
        else if (a.w_bf16)
            add_rmsnorm_typed<bf16_t, bf16_t, float>(a);
        else
            add_rmsnorm_typed<bf16_t, float, double>(a);
    });
}

hipError_t launch_gated_rmsnorm_i8(const NormArgs& all) {
    if (all.rows < 1 || all.rows > GDR_I8_MAX_ROWS || all.heads < 1 || all.heads * all.cols > GDR_NORM_MAX_COLS ||
        (all.cols != 32 && all.cols != 64 && all.cols != 128))
        return hipErrorInvalidValue;
    return by_slices(all, all.heads * all.cols, [](const NormArgs& a) {
        auto w = [&](auto o, auto g) {
            a.w_bf16 ? gated_typed<decltype(o), decltype(g), bf16_t>(a) : gated_typed<decltype(o), decltype(g), float>(a);
        };
        auto g = [&](auto o) { a.gate_bf16 ? w(o, bf16_t{}) : w(o, float{}); };
        a.x_bf16 ? g(bf16_t{}) : g(float{});
    });
}

}  // namespace gdr

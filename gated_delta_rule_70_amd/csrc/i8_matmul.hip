// int8 matrix product with a scale for each row of a and of w:
//   out[m][n] = (sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
// Sums are int32 in the matrix cores (v_mfma_i32_16x16x64_i8), exact for K <= 131071.
#include "i8_launch.h"

#include "gdr_device.h"

namespace gdr {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// D(16x16, int32) += A(16x64) * B(64x16), int8 operands.  Per lane l: A row l % 16 and B column
// l % 16, 16 consecutive reduction bytes of group l / 16 (the same in both); D rows
// 4 (l / 16) .. + 3 of column l % 16.  A is w and B is a throughout, so that a lane holds four
// consecutive columns of one output row.
__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// 16 bytes at p + k, zeros from K on and where the row does not exist.  Any alignment.
__device__ __forceinline__ i32x4 load16(const int8_t* p, int k, int K, bool row) {
    i32x4 v = {0, 0, 0, 0};
    if (!row || k >= K) return v;
    if (k + 16 <= K) {
        __builtin_memcpy(&v, p + k, 16);
        return v;
    }
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (k + i < K) u[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[k + i])) << (8 * (i % 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = static_cast<int>(u[i]);
    return v;
}

// Where the outputs of columns n .. n+3 go: for each column its output's first value of row 0
// and the distance between rows.  Columns of one output share both.
struct Where {
    char* p;  // address of column n in row 0
    int64_t stride;
};
__device__ __forceinline__ Where where(const MatmulOut& o, int n, int elt) {
    char* p = static_cast<char*>(o.ptr[0]);
    int64_t stride = o.stride[0];
    int begin = 0;
#pragma unroll
    for (int i = 1; i < GDR_MATMUL_I8_MAX_OUT; ++i)
        if (i < o.n && n >= o.begin[i]) p = static_cast<char*>(o.ptr[i]), stride = o.stride[i], begin = o.begin[i];
    return Where{p + (int64_t)(n - begin) * elt, stride};
}

template <bool BF16>
__device__ __forceinline__ void store_value(char* p, float x) {
    if constexpr (BF16)
        *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(x);
    else
        *reinterpret_cast<float*>(p) = x;
}

// Columns n .. n+3 of output row m from their sums.
template <bool BF16>
__device__ __forceinline__ void store_quad(const MatmulArgs& g, int m, int n, i32x4 acc) {
    constexpr int E = BF16 ? 2 : 4;
    if (m >= g.M || n >= g.N) return;
    const float sa = g.a_scale[m];
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = min(n + j, g.N - 1);
        v[j] = (float)acc[j] * sa * g.w_scale[c] + (g.bias ? g.bias[c] : 0.f);
    }
    if (g.out.quad && n + 4 <= g.N) {
        const Where to = where(g.out, n, E);
        char* p = to.p + m * to.stride * E;
        if constexpr (BF16)
            *reinterpret_cast<u32x2*>(p) = bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]});
        else
            *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < g.N) {
            const Where to = where(g.out, n + j, E);
            store_value<BF16>(to.p + m * to.stride * E, v[j]);
        }
}

// One workgroup of 4 waves makes 64 x 64 outputs, each wave 32 x 32; 64 reduction bytes at a
// time through LDS.
template <bool BF16>
__global__ __launch_bounds__(256) void matmul_i8_kernel(MatmulArgs g) {
    __shared__ i32x4 sa[64 * 4], sw[64 * 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tiles_n = (g.N + 63) / 64;
    const int m0 = (int)(blockIdx.x / tiles_n) * 64, n0 = (int)(blockIdx.x % tiles_n) * 64;
    const int row = tid >> 2, chunk = tid & 3;
    const int8_t* pa = g.a + (m0 + row) * g.a_stride;
    const int8_t* pw = g.w + (n0 + row) * g.w_stride;
    i32x4 acc[2][2] = {};
    for (int k = 0; k < g.K; k += 64) {
        sa[row * 4 + chunk] = load16(pa, k + chunk * 16, g.K, m0 + row < g.M);
        sw[row * 4 + chunk] = load16(pw, k + chunk * 16, g.K, n0 + row < g.N);
        __syncthreads();
        i32x4 fa[2], fw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fa[i] = sa[((wave >> 1) * 32 + i * 16 + (lane & 15)) * 4 + (lane >> 4)];
            fw[i] = sw[((wave & 1) * 32 + i * 16 + (lane & 15)) * 4 + (lane >> 4)];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma_i8(fw[j], fa[i], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            store_quad<BF16>(g, m0 + (wave >> 1) * 32 + i * 16 + (lane & 15),
                             n0 + (wave & 1) * 32 + j * 16 + (lane >> 4) * 4, acc[i][j]);
}

}  // namespace

hipError_t launch_matmul_i8(const MatmulArgs& g) {
    if (g.M < 1 || g.N < 1 || g.K < 1 || g.K > GDR_MATMUL_I8_MAX_K) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((g.M + 63LL) / 64 * ((g.N + 63) / 64)));
    if (g.out_bf16)
        hipLaunchKernelGGL(matmul_i8_kernel<true>, grid, dim3(256), 0, g.stream, g);
    else
        hipLaunchKernelGGL(matmul_i8_kernel<false>, grid, dim3(256), 0, g.stream, g);
    return hipGetLastError();
}

}  // namespace gdr

// Host-side interface between the entry points of the 8-bit operators (i8_api.cpp) and their
// kernels (i8_norm.hip, i8_matmul.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_i8.h"

namespace gdr {

struct NormArgs {
    int rows, heads, cols;  // heads: 0 for the residual norm
    bool x_bf16, gate_bf16, w_bf16;
    float eps;
    int64_t x_stride, r_stride, out_stride;
    const void *x, *r, *w;  // r: the residual (or NULL), or the gate
    int8_t* q;
    float* scale;
    void* out;  // new residual stream, or NULL
    hipStream_t stream;
};

struct MatmulOut {
    int n;                               // outputs
    int begin[GDR_MATMUL_I8_MAX_OUT + 1];  // first column of each; begin[n] = N
    void* ptr[GDR_MATMUL_I8_MAX_OUT];
    int64_t stride[GDR_MATMUL_I8_MAX_OUT];
};

struct MatmulArgs {
    int M, N, K;
    bool out_bf16;
    int64_t a_stride, w_stride;
    const int8_t *a, *w;
    const float *a_scale, *w_scale, *bias;
    MatmulOut out;
    hipStream_t stream;
};

hipError_t launch_add_rmsnorm_i8(const NormArgs& a);
hipError_t launch_gated_rmsnorm_i8(const NormArgs& a);
hipError_t launch_matmul_i8(const MatmulArgs& a);

}  // namespace gdr

// Host-side interface between the entry points of the layer operators (layer_api.cpp) and their
// kernels (conv.hip, qk_rope.hip, scan.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_layer.h"
#include "scan_plan.h"

namespace gdr {

struct ConvArgs {
    int B, T, D, W;
    int rows;            // of x: B * T, or T of a packed batch
    bool bf16, w_bf16, silu;
    int n_out;
    int begin[GDR_CONV_MAX_OUT + 1];  // first channel of each output; begin[n_out] = D
    void* out[GDR_CONV_MAX_OUT];
    int64_t out_stride[GDR_CONV_MAX_OUT];
    int64_t x_stride;
    const int32_t* cu;   // or NULL
    const void *x, *w, *bias, *state;
    void* out_state;
    hipStream_t stream;
};

struct QkArgs {
    int rows, heads[2], dim, rotated, table_rows, period;
    bool bf16, w_bf16, interleaved, wide_positions;
    float eps;
    int64_t stride[2], out_stride[2];  // of q and k
    const void *in[2], *weight[2];
    void* out[2];
    const float *cos, *sin;
    const void* positions;  // or NULL
    hipStream_t stream;
};

struct ScanArgs {
    int B, T, D, N, G;
    bool bf16, dt_bf16, softplus;
    int64_t x_stride, dt_stride, z_stride, b_stride, c_stride, out_stride;
    const int32_t* cu;  // or NULL
    const void *x, *dt, *z, *b, *c;
    const float *A, *skip, *dt_bias, *h0;
    void* out;
    float* ht;
    int segs, seg_len;  // segments of a sequence (1: it is run whole), and their tokens
    float* workspace;   // segs > 1: B * segs * D * (N + 1) values
    hipStream_t stream;
};

hipError_t launch_causal_conv(const ConvArgs& a);
hipError_t launch_qk_norm_rope(const QkArgs& a);
hipError_t launch_selective_scan(const ScanArgs& a);
hipError_t launch_selective_scan_step(const ScanArgs& a);

// A launch has fewer than 2^32 threads and 2^31 workgroups: `blocks` workgroups of `threads` go in
// slices; launch(first, count) starts one.
template <typename F>
hipError_t by_blocks(int64_t blocks, int threads, F launch) {
    const int64_t most = (int64_t(1) << 31) / threads;
    for (int64_t b = 0; b < blocks; b += most) {
        launch(b, static_cast<unsigned>(blocks - b < most ? blocks - b : most));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gdr

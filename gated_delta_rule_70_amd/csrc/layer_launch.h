// Host-side interface between the entry points of the layer operators (layer_api.cpp) and their
// kernels (conv.hip, qk_rope.hip, scan.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_layer.h"

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

// Segments that the sequences of a scan are cut into, by the sizes alone.
//
// A scan runs a token after the other in workgroups of 16 channels, 25 ns a token for one workgroup on
// a CU and 42 for two.  Where they leave half the CUs idle, segments run side by side: first the states
// behind each from zero, 55 % of a run's work, then each segment from its start.  Two workgroups a CU,
// at 1.55 * 42 ns for each segment's tokens, pay from three segments on, if a sequence is long enough to
// win back the second launch, and segments of 64 tokens or more.  us whole / cut, N = 16: 1 x 511 x 64 15.5 / 9.9,
// 1 x 260 x 64 10.9 / 9.9, 1 x 130 x 64 8.4 / 9.8; two workgroups a CU, 4 x 300 x 256 11.0 / 12.4.
//
// In a packed batch any sequence may have all rows.  Sequence i, from row c on, has the slots from c / seg_len + i
// on: at least as many as segments, and T / seg_len + B in all, whatever the lengths.  Segments pay earlier
// there, since the longest sequence counts: 64 channels, lengths 957, 503, 269, 189 and six short ones 25.6 / 12.2;
// equal lengths may lose, twenty of 600 tokens of 128 channels 20.9 / 32.4, ten of 64 channels 18.6 / 15.5.
struct ScanCut {
    int segs, seg_len;  // packed: segs * B slots
};
inline ScanCut scan_cut(int64_t B, int64_t T, int64_t D, int64_t G, bool packed) {
    const int64_t groups = G * ((D / G + 15) / 16), blocks = B * groups;
    const int64_t n = 512 / blocks, mean = packed ? T / B : T;
    if (n < 3 || mean < (packed ? 128 : 256)) return {1, 0};
    const int64_t len = ((mean + n - 1) / n + 63) / 64 * 64;
    const int64_t segs = packed ? (T / len + 2 * B - 1) / B : (T + len - 1) / len;
    if (segs < 2 || (!packed && T < 512 && segs * blocks > 256)) return {1, 0};
    return {static_cast<int>(segs), static_cast<int>(len)};
}

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

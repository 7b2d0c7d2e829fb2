/*
 * gdr_layer.h -- C ABI of libgdr.so, third part: the operators in front of a recurrence and
 * beside it on AMD Instinct MI355X (gfx950).
 *
 *   gdr_causal_conv          short causal convolution of each channel over time, with SiLU: what
 *                            q, k and v (or a scan's x) pass between projection and recurrence;
 *   gdr_qk_norm_rope         root-mean-square norm of each query and key head and the rotation by
 *                            position, in one pass;
 *   gdr_selective_scan       the recurrence with a diagonal transition that depends on the input
 *                            (a selective state space), over prompts and packed batches;
 *   gdr_selective_scan_step  one token of it for each sequence of a batch, states carried along.
 *
 * Conventions (those of gdr.h unless said otherwise): device pointers; the caller owns every
 * buffer; work is enqueued on `stream` and the call returns without waiting; every argument check
 * runs on the host before any HIP call, so a call that is refused has enqueued nothing (one that
 * returns GDR_ERR_HIP may have); statuses are gdr_status; results are bitwise reproducible (no
 * atomics).  Strides are in elements, between rows (tokens); within a row values are contiguous.
 * Pointers need only their element type's alignment.  "type" is one gdr_dtype (bf16 or fp32) for all
 * tensors named so in a call; bf16 outputs are rounded to nearest even from fp32, once, as they are
 * stored.  Outputs overlap no input and no other output, but for what is said at each call; column
 * ranges of one wider array with rows equally far apart do not overlap.
 *
 * Packed batches: with cu_seqlens (device array [B + 1] of int32, 4-byte aligned) the rows of B
 * sequences lie end to end, sequence i on rows [cu_seqlens[i], cu_seqlens[i + 1]), as in gdr.h:
 * dims B is the number of sequences (at most GDR_VARLEN_MAX_SEQS) and T the rows in all.  Entries are
 * clamped on the device, so no access leaves the tensors whatever they hold, but results are defined
 * only for non-decreasing entries from 0 to T; rows outside [cu_seqlens[0], cu_seqlens[B]) are not
 * written.  A sequence without rows passes its state on.
 */
#ifndef GDR_LAYER_H
#define GDR_LAYER_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDR_LAYER_MAX_ROWS (1 << 30)    /* most rows (tokens) of one call                        */
#define GDR_LAYER_MAX_CHANNELS (1 << 24) /* most channels                                         */
#define GDR_CONV_MAX_OUT 8              /* most separate outputs of one convolution              */
#define GDR_SCAN_MAX_STATES 128         /* most state values of a channel                        */
#define GDR_QK_MAX_DIM 512              /* most values of a head                                 */

#define GDR_CONV_SILU 0x1               /* conv flags: y = silu(sum), else the sum itself        */
#define GDR_SCAN_DT_SOFTPLUS 0x1        /* scan flags: step = softplus(dt + dt_bias)             */
#define GDR_QK_INTERLEAVED 0x1          /* qk flags: pairs (2i, 2i + 1), else (i, i + rotated/2) */

typedef struct {
    int32_t B;            /* sequences, >= 0                                                     */
    int32_t T;            /* tokens of each, or rows in all with cu_seqlens; >= 0                */
    int32_t D;            /* channels, 1 .. GDR_LAYER_MAX_CHANNELS                               */
    int32_t W;            /* taps, 2 .. 4                                                        */
    int32_t dtype;        /* x, state, out_state and outs                                        */
    int32_t weight_dtype; /* weight and bias: that type, or fp32                                 */
    int32_t flags;        /* GDR_CONV_SILU or 0                                                  */
    int32_t n_out;        /* separate outputs, 1 .. GDR_CONV_MAX_OUT                             */
    int32_t out_cols[GDR_CONV_MAX_OUT];   /* channels of each, >= 1; they add up to D            */
    int64_t out_stride[GDR_CONV_MAX_OUT]; /* from one row of each to the next, >= its channels   */
    int64_t x_stride;     /* the same for x, >= 0                                                */
} gdr_conv_dims;

/*
 * For every sequence and channel d, with x[-1], x[-2], ... the last rows of its state (zeros where
 * state is NULL):
 *   s[t]  = bias[d] + sum_j weight[d][j] x[t - (W - 1) + j][d]
 *   y[t]  = s / (1 + exp(-s))  with GDR_CONV_SILU, else s
 * x [B][T][D], weight [D][W], bias [D] (or NULL), state and out_state [B][W - 1][D] dense, oldest row
 * first.  outs[i] (host array of n_out device pointers) receives the i-th group of out_cols[i]
 * channels.  out_state (if not NULL) receives the last W - 1 rows of state and x; it may be state
 * itself.  A single token of every sequence is T = 1.
 */
int gdr_causal_conv(const gdr_conv_dims* dims, const int32_t* cu_seqlens, const void* x, const void* weight,
                    const void* bias, const void* state, void* const* outs, void* out_state, void* stream);

typedef struct {
    int32_t rows;         /* tokens, 0 .. GDR_LAYER_MAX_ROWS                                     */
    int32_t q_heads;      /* >= 1                                                                */
    int32_t k_heads;      /* >= 1; either at most 2^16                                           */
    int32_t dim;          /* values of a head, 1 .. GDR_QK_MAX_DIM                               */
    int32_t rotated;      /* of these, the first that are rotated: even, 0 .. dim                */
    int32_t table_rows;   /* rows of cos and sin, >= 1 (ignored with rotated 0)                  */
    int32_t period;       /* without positions: the position of row r is r % period, >= 1        */
    int32_t position_bits;/* 32 or 64: the type of positions                                     */
    int32_t dtype;        /* q, k and their outputs                                              */
    int32_t weight_dtype; /* weights: that type, or fp32                                         */
    int32_t flags;        /* GDR_QK_INTERLEAVED or 0                                             */
    float eps;            /* finite, >= 0                                                        */
    int64_t q_stride, k_stride;         /* from one row to the next, >= 0                        */
    int64_t out_q_stride, out_k_stride; /* the same, >= heads * dim                              */
} gdr_qk_dims;

/*
 * For every row and head, with n = x / sqrt(mean(x^2) + eps) * weight (weight NULL: without it) and
 * c, s the row of the tables at the row's position:
 *   (a, b) -> (a c_i - b s_i, b c_i + a s_i)  for the pair (a, b) = (n[i], n[i + rotated / 2]), or
 *   (n[2 i], n[2 i + 1]) with GDR_QK_INTERLEAVED, i < rotated / 2; the other values are n's.
 * q [rows][q_heads][dim], k [rows][k_heads][dim] (the heads of a row contiguous); cos and sin
 * [table_rows][rotated / 2] fp32, dense; positions [rows] of int32 or int64, or NULL.  The rotated
 * values of a row whose position lies outside the tables are NaN.  A head of zeros stays zero, with
 * eps = 0 too; one that holds NaN or infinity is NaN throughout.  out_q may be q itself and out_k k
 * (same pointer and stride).
 */
int gdr_qk_norm_rope(const gdr_qk_dims* dims, const void* q, const void* k, const void* q_weight,
                     const void* k_weight, const float* cos, const float* sin, const void* positions, void* out_q,
                     void* out_k, void* stream);

typedef struct {
    int32_t B;            /* sequences, >= 0                                                     */
    int32_t T;            /* tokens of each, or rows in all with cu_seqlens; >= 0.  Step: 1      */
    int32_t D;            /* channels, 1 .. GDR_LAYER_MAX_CHANNELS                               */
    int32_t N;            /* state values of a channel, 1 .. GDR_SCAN_MAX_STATES                 */
    int32_t G;            /* groups of channels that share B and C, D % G == 0                   */
    int32_t dtype;        /* x, z, B, C and out                                                  */
    int32_t dt_dtype;     /* dt: that type, or fp32                                              */
    int32_t flags;        /* GDR_SCAN_DT_SOFTPLUS or 0                                           */
    int64_t x_stride, dt_stride, z_stride; /* from one row to the next, >= 0                     */
    int64_t b_stride, c_stride;            /* the same                                           */
    int64_t out_stride;                    /* the same, >= D                                     */
} gdr_scan_dims;

/*
 * For every sequence and channel d (group d / (D / G)), the state h[N] from h0 (zeros where NULL):
 *   step   = dt[t][d] + dt_bias[d], or softplus of it with GDR_SCAN_DT_SOFTPLUS
 *   h[n]   = exp(step A[d][n]) h[n] + step x[t][d] B[t][n]
 *   y      = sum_n C[t][n] h[n] + Dskip[d] x[t][d]
 *   out    = y z[t][d] / (1 + exp(-z[t][d])), or y where z is NULL
 * x, dt, z, out [B][T][D]; B and C [B][T][G][N] (a row's groups contiguous); A [D][N], Dskip and
 * dt_bias [D] fp32, dense (these two may be NULL); h0 and ht [B][D][N] fp32, dense.  States are fp32
 * throughout.  ht (if not NULL) receives the last state; it may be h0 itself.  A is expected not
 * to be positive; where it is, the state grows as the formula says (a token's factor past fp32's
 * range is infinity, and NaN on a state of zero, or in a call that needs a workspace on any state).
 * Infinite inputs and states give what the formula gives, but that what lies below fp32's normal range
 * counts as zero: infinity times such a factor of a token, or such a gate, is NaN.  Infinities in A count as the
 * finite values next to them (-infinity: a state that each token of a positive step begins anew).
 */
int gdr_selective_scan(const gdr_scan_dims* dims, const int32_t* cu_seqlens, const void* x, const void* dt,
                       const float* A, const void* B, const void* C, const float* Dskip, const void* z,
                       const float* dt_bias, const float* h0, void* out, float* ht, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace gdr_selective_scan needs for these dims, `packed` saying whether the call
 * has cu_seqlens (0 for most dims, and for invalid ones; then `workspace` may be NULL).  Long sequences
 * of few channels are cut into segments that run side by side; the workspace, 4-byte aligned, holds the
 * state behind each.  Its contents on entry are ignored; calls that overlap in time need one each.
 */
size_t gdr_selective_scan_workspace_bytes(const gdr_scan_dims* dims, int packed);

/* One token for each of B sequences (T must be 1): the same formulas, each state value read once
 * and written once.  Normally called in place (ht == h0). */
int gdr_selective_scan_step(const gdr_scan_dims* dims, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const float* Dskip, const void* z, const float* dt_bias,
                            const float* h0, void* out, float* ht, void* stream);

#ifdef __cplusplus
}
#endif
#endif

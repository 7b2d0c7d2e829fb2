/*
 * gdr_i8.h -- C ABI of libgdr.so, second part: the 8-bit projections around a gated delta
 * rule layer on AMD Instinct MI355X (gfx950).
 *
 * The calls of gdr.h take q, k, v, g and beta that a projection has made, and give an o that
 * the next projection reads.  These are the three operators in between, with activations and
 * weights in 8-bit integers:
 *
 *   gdr_add_rmsnorm_i8    residual addition, root-mean-square norm, int8 codes and a scale for
 *                         each row: the input of a projection;
 *   gdr_matmul_i8         int8 matrix product with a scale for each row (token) and each
 *                         weight row (output channel), its columns cut into separate dense
 *                         outputs (q, k, v, ... from one product);
 *   gdr_gated_rmsnorm_i8  norm per value head, times silu(gate), int8 codes and a scale for
 *                         each token: from the delta rule's o to the output projection.
 *
 * Conventions (those of gdr.h unless said otherwise): device pointers; the caller owns every
 * buffer; work is enqueued on `stream` and the call returns without waiting; every argument
 * check runs on the host before any HIP call, so a call that is refused has enqueued nothing
 * (one that returns GDR_ERR_HIP may have); statuses are gdr_status; results are bitwise
 * reproducible (no atomics).  rows == 0 is a valid call that does nothing (pointers may then be
 * NULL).  Strides are in elements, between rows; within a row values are contiguous.  Pointers
 * need only their element type's alignment; the product is fastest where a, w and their row
 * strides are multiples of 128 bytes, then of 4.  It reads the aligned words of 4 bytes that hold
 * an operand's first and last bytes whole.
 */
#ifndef GDR_I8_H
#define GDR_I8_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDR_I8_MAX_ROWS (1 << 30)    /* most rows (tokens) of one call                       */
#define GDR_NORM_MAX_COLS 32768      /* most values in one row (heads * cols) of the norms    */
#define GDR_MATMUL_I8_MAX_K 131071   /* longest reduction: 128 * 128 * K stays below 2^31     */
#define GDR_MATMUL_I8_MAX_OUT 8      /* most separate outputs of one product                  */

/* Dims of the two norms. */
typedef struct {
    int32_t rows;         /* tokens, 0 .. GDR_I8_MAX_ROWS                                   */
    int32_t heads;        /* gdr_gated_rmsnorm_i8: value heads; gdr_add_rmsnorm_i8: 1         */
    int32_t cols;         /* values per row, or per head (then 32, 64 or 128)                 */
    int32_t x_dtype;      /* x, residual and out_residual, or o (gdr_dtype)                   */
    int32_t gate_dtype;   /* gate; ignored by gdr_add_rmsnorm_i8                              */
    int32_t weight_dtype; /* weight: fp32, or bf16 (with gdr_add_rmsnorm_i8 only for bf16 x)  */
    float eps;            /* finite, >= 0                                                     */
    int64_t x_stride;     /* elements from one row of x (o) to the next, >= 0                 */
    int64_t r_stride;     /* the same for residual (gate), >= 0                               */
    int64_t out_stride;   /* the same for out_residual, >= cols                               */
} gdr_norm_dims;

/*
 * For each row, with r = 0 where residual is NULL:
 *   s   = x + r, rounded to x_dtype                        -> out_residual (if not NULL)
 *   t   = s * weight,  A = max |t|,  rho = 1 / sqrt(mean(s^2) + eps)
 *   q   = rint(127 t / A) (ties to even)                   -> q      [rows][cols] int8, dense
 *   A * rho / 127                                          -> scale  [rows]       fp32
 * so that q * scale is the normed row to 8 bits.  q does not depend on rho; it is the code of
 * the exact quotient (borders between two codes are decided in 64 bits).  A row with A = 0
 * has q = 0 and scale 0.  A row whose t holds a NaN, an infinity or a value beyond fp32's
 * range has q = 0 and scale NaN.  out_residual may be x or residual itself (same pointer and
 * stride), or a column range beside theirs in one wider array; no other output may overlap an input
 * or another output.
 */
int gdr_add_rmsnorm_i8(const gdr_norm_dims* dims, const void* x, const void* residual, const void* weight,
                       int8_t* q, float* scale, void* out_residual, void* stream);

/*
 * For each token, over its heads h and values v (o, gate [rows][heads][cols], the heads of a
 * row contiguous; weight [cols]):
 *   n   = o / sqrt(mean_v(o^2) + eps) * weight_v * gate / (1 + exp(-gate))
 *   A   = max |n| over the token
 *   q   = rint(127 n / A)                                  -> q      [rows][heads*cols] int8
 *   A / 127                                                -> scale  [rows]             fp32
 * n is computed in fp32 (sums of squares in fp64), so a value within fp32 rounding of the
 * border between two codes may take either, and a gate below -87, where silu is less than 1e-35,
 * may count as closed.  The range is fp32's too: weight times silu counts as infinite beyond it,
 * and a token of nothing above 1e-38 has the bits that fp32 has there.  Empty and non-finite rows
 * as above.
 * out_stride is ignored.
 */
int gdr_gated_rmsnorm_i8(const gdr_norm_dims* dims, const void* o, const void* gate, const void* weight,
                         int8_t* q, float* scale, void* stream);

/* Dims of the product. */
typedef struct {
    int32_t M;            /* rows of a (tokens), 0 .. GDR_I8_MAX_ROWS                         */
    int32_t K;            /* 1 .. GDR_MATMUL_I8_MAX_K                                         */
    int32_t n_out;        /* separate outputs, 1 .. GDR_MATMUL_I8_MAX_OUT                     */
    int32_t out_dtype;    /* gdr_dtype of every output                                        */
    int32_t out_cols[GDR_MATMUL_I8_MAX_OUT];  /* columns of each, >= 1; their sum is N, at most
                             2^30, and M / 256 * N / 256 (each rounded up) below 2^23         */
    int64_t out_stride[GDR_MATMUL_I8_MAX_OUT];/* elements between rows of each, >= its columns*/
    int64_t a_stride;     /* bytes from one row of a to the next, >= 0                        */
    int64_t w_stride;     /* bytes from one row of w to the next, >= 0                        */
} gdr_matmul_i8_dims;

/*
 *   out[m][n] = (sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
 * a [M][K] int8, w [N][K] int8, a_scale [M], w_scale [N] and bias [N] fp32 (bias may be NULL).
 * The sum is exact in int32 (any int8 values, -128 among them); scales and bias are applied in
 * fp32; bf16 outputs are rounded to nearest even as they are stored.  outs[i] (host array of
 * n_out device pointers) receives the i-th group of out_cols[i] columns.
 */
int gdr_matmul_i8(const gdr_matmul_i8_dims* dims, const int8_t* a, const float* a_scale, const int8_t* w,
                  const float* w_scale, const float* bias, void* const* outs, void* stream);

#ifdef __cplusplus
}
#endif
#endif

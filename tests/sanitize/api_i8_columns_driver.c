/* Column ranges of one wider array as operands of the 8-bit operators (i8_api.cpp, launchers stubbed
 * out, fake device addresses): accepted where no byte is shared, GDR_ERR_ALIAS one element nearer.
 * An accepted call reaches the stub, which reports GDR_ERR_HIP. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdr_i8.h"

static int fails = 0;
#define SAME(got, want)                                                                       \
    do {                                                                                      \
        int g_ = (got);                                                                       \
        if (g_ != (want)) {                                                                   \
            fprintf(stderr, "line %d: %s is %d, not %s\n", __LINE__, #got, g_, #want);        \
            ++fails;                                                                          \
        }                                                                                     \
    } while (0)

#define P(i, off) ((void*)(uintptr_t)((1ull << 40) + (uint64_t)(i) * (1ull << 36) + (off)))

/* x at 0, residual at r and the new stream at o of one array with rows `stride` values apart, of 64
 * values of e bytes each. */
static int norm(int64_t rows, int64_t r, int64_t o, int64_t stride, int64_t o_stride, int e) {
    gdr_norm_dims d = {(int32_t)rows, 1, 64, e == 4, 0, e == 4, 1e-6f, stride, stride, o_stride};
    return gdr_add_rmsnorm_i8(&d, P(0, 0), P(0, r * e), P(1, 0), P(2, 0), P(3, 0), P(0, o * e), NULL);
}

/* two outputs of 32 and 16 fp32 values at 0 and `at` */
static int product(int64_t rows, int64_t at, int64_t stride, int64_t stride2) {
    gdr_matmul_i8_dims d;
    memset(&d, 0, sizeof d);
    d.M = (int32_t)rows, d.K = 64, d.n_out = 2, d.out_dtype = GDR_F32, d.a_stride = 64, d.w_stride = 64;
    d.out_cols[0] = 32, d.out_cols[1] = 16, d.out_stride[0] = stride, d.out_stride[1] = stride2;
    void* outs[2] = {P(4, 0), P(4, at * 4)};
    return gdr_matmul_i8(&d, P(0, 0), P(1, 0), P(2, 0), P(3, 0), NULL, outs, NULL);
}

int main(void) {
    for (int e = 2; e <= 4; e += 2)
        for (int64_t rows = 2; rows < 9; rows += 3) {
            /* x | residual | new stream, in any order, edge to edge */
            SAME(norm(rows, 64, 128, 192, 192, e), GDR_ERR_HIP);
            SAME(norm(rows, 128, 64, 192, 192, e), GDR_ERR_HIP);
            SAME(norm(rows, 0, 64, 128, 128, e), GDR_ERR_HIP);
            SAME(norm(rows, 0, -64, 128, 128, e), GDR_ERR_HIP);
            SAME(norm(rows, 0, 64 + 128, 128, 128, e), GDR_ERR_HIP); /* a row further down */
            /* one element nearer, on either side */
            SAME(norm(rows, 64, 127, 192, 192, e), GDR_ERR_ALIAS);
            SAME(norm(rows, 128, 63, 192, 192, e), GDR_ERR_ALIAS);
            SAME(norm(rows, 128, 65, 192, 192, e), GDR_ERR_ALIAS);
            SAME(norm(rows, 0, 63, 128, 128, e), GDR_ERR_ALIAS);
            SAME(norm(rows, 0, 65, 128, 128, e), GDR_ERR_ALIAS); /* into the next row */
            SAME(norm(rows, 0, -63, 128, 128, e), GDR_ERR_ALIAS);
            SAME(norm(rows, 0, 64, 128, 130, e), GDR_ERR_ALIAS); /* rows not equally far apart */
            SAME(norm(rows, 0, 128, 128, 128, e), GDR_ERR_ALIAS); /* its own columns, a row further down */
            /* in place, as ever */
            SAME(norm(rows, 64, 0, 128, 128, e), GDR_ERR_HIP);
            SAME(norm(rows, 64, 64, 128, 128, e), GDR_ERR_HIP);
        }
    SAME(norm(1, 64, 128, 0, 192, 2), GDR_ERR_HIP);
    SAME(norm(1, 64, 127, 192, 192, 2), GDR_ERR_ALIAS);
    for (int64_t rows = 2; rows < 9; rows += 3) {
        SAME(product(rows, 32, 48, 48), GDR_ERR_HIP);
        SAME(product(rows, 31, 48, 48), GDR_ERR_ALIAS);
        SAME(product(rows, 33, 48, 48), GDR_ERR_ALIAS);
        SAME(product(rows, 32, 48, 50), GDR_ERR_ALIAS);
        SAME(product(rows, -16, 48, 48), GDR_ERR_HIP);
        SAME(product(rows, -17, 48, 48), GDR_ERR_ALIAS);
        SAME(product(rows, -15, 48, 48), GDR_ERR_ALIAS);
        SAME(product(rows, 0, 48, 48), GDR_ERR_ALIAS);
    }
    SAME(product(1, 32, 32, 16), GDR_ERR_HIP);
    SAME(product(1, 31, 48, 48), GDR_ERR_ALIAS);
    if (fails) return 1;
    puts("i8 columns ok");
    return 0;
}

/* Drives the host entry points of the 8-bit operators (i8_api.cpp, launchers stubbed out) under
 * host sanitizers: random dims from ordinary to extreme, on fake device addresses that no call
 * dereferences.  Every call must end with a documented status. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdr_i8.h"

static int fails = 0;
#define CHECK(cond)                                                                     \
    do {                                                                                \
        if (!(cond)) {                                                                  \
            fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__);          \
            ++fails;                                                                    \
        }                                                                               \
    } while (0)

#define P(i) ((void*)(uintptr_t)((1ull << 40) + (uint64_t)(i) * (1ull << 36)))

static uint64_t state = 88172645463325252ull;
static uint64_t rnd(void) {
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
static int64_t pick(const int64_t* v, int n) { return v[rnd() % (uint64_t)n]; }
#define PICK(...) pick((const int64_t[]){__VA_ARGS__}, (int)(sizeof((int64_t[]){__VA_ARGS__}) / sizeof(int64_t)))
#define BIG INT64_MAX
#define STRIDE PICK(0, 1, 64, 128, 4096, 4096, 5000, 1ll << 31, 1ll << 40, 1ll << 61, BIG, -1)
#define ROWS PICK(0, 1, 1, 2, 7, 4097, 1 << 20, INT32_MAX, -1)

static int known(int s) { return (s >= GDR_OK && s <= GDR_ERR_ALIAS) || s == GDR_ERR_HIP; }

int main(void) {
    int reached = 0;
    for (int i = 0; i < 400000; ++i) {
        gdr_norm_dims d = {(int32_t)ROWS, (int32_t)PICK(1, 1, 1, 2, 32, 0, INT32_MAX), (int32_t)PICK(1, 32, 64, 128, 4096, 32768, 32769, INT32_MAX, 0),
                           (int32_t)PICK(0, 1, 2), (int32_t)PICK(0, 1, 2), (int32_t)PICK(0, 1, 3), 1e-6f, STRIDE, STRIDE, STRIDE};
        void* x = P(PICK(0, 0, 1));
        void* out = rnd() % 3 ? P(PICK(5, 5, 0, 1)) : NULL;
        int a = gdr_add_rmsnorm_i8(&d, x, rnd() % 2 ? P(1) : NULL, P(2), P(3), P(4), out, NULL);
        int b = gdr_gated_rmsnorm_i8(&d, x, P(1), P(2), P(3), P(4), NULL);
        CHECK(known(a) && known(b));
        reached += (a == GDR_ERR_HIP) + (b == GDR_ERR_HIP);
    }
    CHECK(reached > 1000);
    reached = 0;
    for (int i = 0; i < 400000; ++i) {
        gdr_matmul_i8_dims d;
        memset(&d, 0, sizeof d);
        d.M = (int32_t)ROWS;
        d.K = (int32_t)PICK(1, 64, 4096, 131071, 131072, 0, INT32_MAX);
        d.n_out = (int32_t)PICK(1, 1, 2, 3, 8, 9, 0, -1);
        d.out_dtype = (int32_t)PICK(0, 1, 1, 0, 2);
        for (int j = 0; j < GDR_MATMUL_I8_MAX_OUT; ++j) {
            d.out_cols[j] = (int32_t)PICK(1, 4, 64, 64, 1000, 4096, INT32_MAX, 0);
            d.out_stride[j] = STRIDE;
        }
        d.a_stride = STRIDE;
        d.w_stride = STRIDE;
        void* outs[GDR_MATMUL_I8_MAX_OUT];
        for (int j = 0; j < GDR_MATMUL_I8_MAX_OUT; ++j) outs[j] = (char*)P(rnd() % 8 ? 10 + j : 10) + PICK(0, 0, 128, 2, 1);
        int s = gdr_matmul_i8(&d, P(0), P(1), P(2), P(3), rnd() % 2 ? P(4) : NULL, outs, NULL);
        CHECK(known(s));
        reached += s == GDR_ERR_HIP;
    }
    CHECK(reached > 500);
    if (fails) return 1;
    puts("i8 api sanitize ok");
    return 0;
}

/* Drives the host entry points of the layer operators (layer_api.cpp, launchers stubbed out) under
 * host sanitizers: random dims from ordinary to extreme, on fake device addresses that no call
 * dereferences.  Every call must end with a documented status. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdr_layer.h"

static int fails = 0;
#define CHECK(cond)                                                                     \
    do {                                                                                \
        if (!(cond)) {                                                                  \
            fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__);          \
            ++fails;                                                                    \
        }                                                                               \
    } while (0)

#define P(i) ((void*)(uintptr_t)((1ull << 40) + (uint64_t)(i) * (1ull << 38)))

static uint64_t state = 88172645463325252ull;
static uint64_t rnd(void) {
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
static int64_t pick(const int64_t* v, int n) { return v[rnd() % (uint64_t)n]; }
#define PICK(...) pick((const int64_t[]){__VA_ARGS__}, (int)(sizeof((int64_t[]){__VA_ARGS__}) / sizeof(int64_t)))
#define STRIDE PICK(0, 64, 128, 4096, 4096, 4096, 5000, 1ll << 31, 1ll << 40, 1ll << 61, INT64_MAX, -1)
#define ROWS PICK(0, 1, 1, 2, 7, 4097, 1 << 20, INT32_MAX, -1)
#define CHANNELS PICK(1, 64, 64, 96, 4096, 1 << 24, (1 << 24) + 1, INT32_MAX, 0, -1)
#define MAYBE(p) (rnd() % 4 ? (p) : NULL)

static int known(int s) { return s >= GDR_OK && s <= GDR_ERR_HIP; }

int main(void) {
    int reached[4] = {0, 0, 0, 0};
    for (int i = 0; i < 400000; ++i) {
        gdr_conv_dims d;
        memset(&d, 0, sizeof d);
        d.B = (int32_t)ROWS, d.T = (int32_t)ROWS, d.D = (int32_t)CHANNELS;
        d.W = (int32_t)PICK(2, 3, 4, 4, 5, 0, INT32_MAX);
        d.dtype = (int32_t)PICK(0, 0, 1, 2), d.weight_dtype = (int32_t)PICK(0, 1, 1, 3);
        d.flags = (int32_t)PICK(0, 1, 1, 2), d.n_out = (int32_t)PICK(1, 1, 2, 8, 9, 0, -1);
        void* outs[GDR_CONV_MAX_OUT];
        for (int j = 0; j < GDR_CONV_MAX_OUT; ++j) {
            d.out_cols[j] = d.n_out == 1 ? d.D : (int32_t)PICK(32, 32, 64, 4096, INT32_MAX, 0);
            d.out_stride[j] = STRIDE;
            outs[j] = MAYBE(P(10 + j));
        }
        d.x_stride = STRIDE;
        const int s = gdr_causal_conv(&d, rnd() % 3 ? NULL : P(9), MAYBE(P(0)), MAYBE(P(1)), MAYBE(P(2)), MAYBE(P(3)),
                                      rnd() % 16 ? outs : NULL, MAYBE(P(PICK(3, 4, 4, 0))), NULL);
        CHECK(known(s));
        reached[0] += s == GDR_ERR_HIP;

        gdr_qk_dims q = {(int32_t)ROWS, (int32_t)PICK(1, 4, 32, 65536, 0, INT32_MAX), (int32_t)PICK(1, 4, 8, 65536, -1),
                         (int32_t)PICK(1, 64, 128, 512, 513, 0, INT32_MAX), (int32_t)PICK(0, 2, 32, 64, 63, -2, INT32_MAX),
                         (int32_t)PICK(1, 4096, INT32_MAX, 0, -1), (int32_t)PICK(1, 4097, 0, INT32_MAX),
                         (int32_t)PICK(32, 64, 16), (int32_t)PICK(0, 1, 2), (int32_t)PICK(0, 1, 1, 3), (int32_t)PICK(0, 1, 2),
                         1e-6f, STRIDE, STRIDE, STRIDE, STRIDE};
        const int t = gdr_qk_norm_rope(&q, MAYBE(P(0)), MAYBE(P(1)), MAYBE(P(2)), MAYBE(P(3)), MAYBE(P(4)), MAYBE(P(5)),
                                       MAYBE(P(6)), MAYBE(P(PICK(7, 0, 7, 1))), MAYBE(P(PICK(8, 1, 8, 0))), NULL);
        CHECK(known(t));
        reached[1] += t == GDR_ERR_HIP;

        for (int step = 0; step < 2; ++step) {
            gdr_scan_dims c = {(int32_t)ROWS, step && rnd() % 8 ? 1 : (int32_t)ROWS, (int32_t)CHANNELS,
                               (int32_t)PICK(1, 16, 16, 128, 129, 0, INT32_MAX), (int32_t)PICK(1, 1, 2, 7, 0, -1, INT32_MAX),
                               (int32_t)PICK(0, 0, 1, 2), (int32_t)PICK(0, 1, 1, 2), (int32_t)PICK(0, 1, 2), STRIDE, STRIDE,
                               STRIDE, STRIDE, STRIDE, STRIDE};
            float* h0 = MAYBE(P(PICK(8, 8, 0)));
            float* ht = MAYBE(P(PICK(8, 9, 9, 2)));
            const void *x = MAYBE(P(0)), *dt = MAYBE(P(1)), *B = MAYBE(P(3)), *C = MAYBE(P(4)), *z = MAYBE(P(6));
            const float *A = MAYBE(P(2)), *skip = MAYBE(P(5)), *bias = MAYBE(P(7));
            void* out = MAYBE(P(PICK(10, 10, 6)));
            void* ws = MAYBE(P(PICK(12, 12, 3)));
            (void)gdr_selective_scan_workspace_bytes(&c, step);
            const int u = step ? gdr_selective_scan_step(&c, x, dt, A, B, C, skip, z, bias, h0, out, ht, NULL)
                               : gdr_selective_scan(&c, rnd() % 3 ? NULL : P(11), x, dt, A, B, C, skip, z, bias, h0, out, ht, ws,
                                                    (size_t)PICK(0, 1 << 20, INT64_MAX), NULL);
            CHECK(known(u));
            reached[2 + step] += u == GDR_ERR_HIP;
        }
    }
    for (int i = 0; i < 4; ++i) {
        printf("reached %d\n", reached[i]);
        CHECK(reached[i] > 100);
    }
    CHECK(gdr_causal_conv(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == GDR_ERR_NULL);
    if (!fails) printf("layer api sanitize ok\n");
    return fails != 0;
}

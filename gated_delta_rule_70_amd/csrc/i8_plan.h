// Which kernels a product runs on (i8_matmul.hip): host arithmetic only, without HIP.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace gdr {

struct Operands {
    uint64_t a, w;  // addresses
    int M, N, K;
    int64_t a_stride, w_stride;
};
// Where rows of a and w begin: all at whole lines of 128 bytes (0), at multiples of 16 (1), at
// whole words (2), or anywhere (3).
inline int places_of(const Operands& g) {
    const uint64_t all = g.a | g.w | (g.M > 1 ? (uint64_t)g.a_stride : 0) | (g.N > 1 ? (uint64_t)g.w_stride : 0);
    return all % 128 == 0 ? 0 : all % 16 == 0 ? 1 : all % 4 == 0 ? 2 : 3;
}

// A tile's rows lie within 2^31 bytes.
inline bool near(int64_t stride, int rows, int K) { return rows == 1 || stride <= (INT32_MAX - K - 8) / 255; }

// Form of a product and its expected time, from how many tiles a CU of the 256 gets (past four of
// them the CUs no longer keep step, and a fraction counts) and what a tile takes: a fixed part
// (filling the pipeline, storing) and a part for each reduction byte.  Forms of which several
// workgroups fit a CU overlap their fixed parts; the others slow down as more CUs draw on memory
// and power.  Where rows do not begin at whole lines, the 128 bytes of a stage lie in two lines and
// all forms but those that read 256 or more in a row take longer; fragments that have to be moved into
// place cost more again.  The constants were fitted to 11000 random sizes (17 to 32768 rows, 128 to
// 12288 columns, reductions of 256 to 8192), on operands that stay in the last-level cache; the form so
// chosen takes 0.6 % longer than the fastest on average, 14 % at the 99th percentile.  Below 17 rows
// they are carried on, with one factor for rows of a that the first form reads once, set on single rows
// of 4096 and 12288 columns.
// M x N x K in us from one call to the next, rows beginning at whole lines; operands in the last-level
// cache / from memory:
//                           32x64        128x64     128x128 deep     128x128       192x256       256x256
//      32 x 12288 x 4096  11.0 / 15.4  12.6 / 18.8  15.1 / 20.5  22.1 / 31.4   32.0 / 40.9   37.8 / 48.1
//     128 x  4096 x 4096   8.7 / 11.4  12.8 / 18.5  15.8 / 22.7  22.4 / 31.7   33.0 / 44.5   39.0 / 48.7
//     512 x  4096 x 4096  22.3 / 28.5  14.1 / 18.3  16.4 / 22.1  22.7 / 31.4   33.7 / 45.1   40.3 / 52.4
//    1024 x  4096 x 4096  43.6 / 55.0  23.1 / 28.4  20.5 / 23.8  24.4 / 32.6   34.4 / 43.5   40.9 / 52.9
//     512 x 12288 x 4096  56.7 / 77.2  34.0 / 43.8               28.7 / 40.9   35.6 / 47.1   41.6 / 54.1
//    2048 x  4096 x 4096  86.8 / 98.4  43.6 / 51.4               34.2 / 39.2   36.9 / 48.0   42.1 / 54.9
//    4096 x  4096 x 1024  67.9 / 72.9  29.9 / 37.8               24.4 / 29.7   28.6 / 31.1   21.5 / 24.1
//    8192 x  8192 x  512                101 /  104               78.6 / 78.4   62.9 / 64.9   72.4 / 72.1
//    1691 x  5760 x 4096  99.1 /  107  53.5 / 61.5               52.3 / 64.2   38.8 / 46.8   42.2 / 52.6
//    3000 x  4096 x 4096   125 /  131  64.5 / 70.6               54.4 / 59.1   43.3 / 51.2   45.3 / 56.0
//    8192 x  2048 x 8192   324 /  332   181 /  183                132 /  135    142 /  151    109 /  109
// Fewer outputs:            16x16        32x32        32x64
//       1 x  4096 x 4096   5.5 /  6.2   6.2 /  8.3   7.9 / 10.3
//       1 x 12288 x 4096  10.0 / 12.2               10.3 / 14.1
//       2 x 12288 x 4096  10.2 / 12.4               10.4 / 14.1
//      16 x  8192 x 4096   9.9 / 12.5   8.4 / 10.3   8.4 / 13.1
//      64 x  4096 x 4096  16.9 / 17.4   6.9 /  9.2   8.4 / 11.4
//     178 x  1280 x 3712  15.7 / 16.0   6.6 /  7.3   8.4 /  9.0
//     256 x  1024 x 8192  30.7 / 31.1   9.1 / 11.7  12.5 / 16.8
// 32x32 tiles serve where each CU has at most one: 3900 random sizes of that kind take 6 to 10 %
// longer without them (the form chosen 0.6 % longer than the fastest).
constexpr int64_t kMostTiles = (1 << 23) - 1;  // a launch has fewer than 2^32 threads, 512 for each tile
enum class Form { rows, t32x32, t32x64, t128x64, t128x128_deep, t128x128, t192x256, t256x256 };
struct Plan {
    Form form;
    double us;
};
struct Cost {
    uint32_t rows, cols;      // of a tile
    int a_cu;                 // workgroups that fit a CU
    double fixed, per_k;      // us for a tile, and for 1000 reduction bytes of it
    double more;              // added to per_k: for a CU's first tile (several a CU), once every CU has one (one a CU)
    double places[4];         // per_k for each of places_of(), in relation to the first
};
constexpr Cost kCosts[] = {{16, 16, 4, 1.0, .85, 0, {1, .72, .82, 1.42}},
                           {32, 32, 1, 2.3, .53, .27, {1, 1.17, 1.18, 1.75}},
                           {32, 64, 2, 2.6, 1.25, 0, {1, 1.02, 1.11, 1.54}},
                           {128, 64, 2, 2.7, 2.34, 0, {1, 1.51, 1.57, 2.50}},
                           {128, 128, 1, 3.5, 2.5, .9, {1, 1.60, 1.72, 0}},  // four stages: not where fragments are moved
                           {128, 128, 2, 4.4, 3.3, .5, {1, 1.41, 1.49, 2.05}},
                           {192, 256, 1, 7.3, 7.3, 1.2, {1, 1.32, 1.37, 1.90}},
                           {256, 256, 1, 9.9, 8.1, 1.6, {1, 1.38, 1.35, 1.95}}};
inline Plan plan(uint32_t M, uint32_t N, int K, int places) {
    Plan best{Form::rows, 1e30};
    for (int f = 0; f < 8; ++f) {
        const Cost& c = kCosts[f];
        const int64_t tiles = (int64_t)((M + c.rows - 1) / c.rows) * ((N + c.cols - 1) / c.cols);
        if (tiles > kMostTiles || ((f == (int)Form::t32x32 || f == (int)Form::t128x128_deep) && tiles > 256) ||
            (f == (int)Form::t128x128_deep && places == 3))
            continue;
        double k = K * 1e-3 * c.places[places];
        if (f == (int)Form::rows && M < 16) k *= .6 + .025 * M;  // rows of a that are read once
        const double n = tiles <= 1024 ? (double)((tiles + 255) / 256) : tiles / 256. + .5;
        const double fill = std::min(1.0, tiles / 256.0);
        const double groups = tiles <= 1024 ? (double)((tiles + 256 * c.a_cu - 1) / (256 * c.a_cu)) : n / c.a_cu + .5;
        const double us = c.a_cu > 1 ? c.fixed * groups + k * (c.per_k * n + c.more)
                                        : n * (c.fixed + k * (c.per_k + c.more * fill * fill));
        if (2.0 + us < best.us) best = Plan{(Form)f, 2.0 + us};  // 2: a launch
    }
    return best;
}

// The launches of a product, in order: f(first row, rows, form, whether fragments are moved into
// place) for each, until one returns false.
template <typename F>
bool launches(const Operands& g, int first, F f) {
    auto rows_of = [&](int at, int count) {
        Operands r = g;
        r.M = count;
        r.a += (uint64_t)(at * g.a_stride);
        return r;
    };
    auto one = [&](Form form, int at, int count) { return f(first + at, count, form, places_of(rows_of(at, count)) == 3); };
    const int places = places_of(g);
    if (!near(g.a_stride, g.M, g.K) || !near(g.w_stride, g.N, g.K)) {
        // rows this far apart: the forms that address each row by itself
        if ((g.M + 31LL) / 32 * ((g.N + 63LL) / 64) > kMostTiles) {
            const int half = g.M / 2;
            return half > 0 && launches(rows_of(0, half), first, f) && launches(rows_of(half, g.M - half), first + half, f);
        }
        const Form form = plan(g.M, g.N, g.K, places).form;
        return one(form == Form::rows || form == Form::t32x32 ? form : Form::t32x64, 0, g.M);
    }
    const Plan whole = plan(g.M, g.N, g.K, places);
    // Rows that would cost a round of large tiles of their own go into a second launch, of smaller
    // ones: those past a multiple of 256 (4097 x 12288 x 4096: 189 against 207 us), or past the last
    // round in which every CU has a tile (6023 x 2692 x 7008: 134 against 185).  Where less than a
    // seventh is expected to be saved the two launches were as often slower.
    const int high = g.M / 256, wide = (g.N + 255) / 256;
    const int heads[2] = {high * 256, (int)((int64_t)high * wide / 256 * 256 / wide * 256)};
    Plan first_plan{}, second{};
    int head = 0;
    double least = .85 * whole.us;
    for (int h : heads) {
        if (h < 1 || h >= g.M) continue;
        const Plan a = plan(h, g.N, g.K, places), b = plan(g.M - h, g.N, g.K, places);
        if (a.us + b.us < least) least = a.us + b.us, head = h, first_plan = a, second = b;
    }
    if (head > 0) return one(first_plan.form, 0, head) && one(second.form, head, g.M - head);
    return one(whole.form, 0, g.M);
}

}  // namespace gdr

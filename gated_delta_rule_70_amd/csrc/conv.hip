// Short causal convolution of each channel over time (gdr_causal_conv).
//
// y[t][d] = act(bias[d] + sum_j w[d][j] x[t - (W - 1) + j][d]).  Each thread takes a tile of rows of eight
// channels: it loads them and the W - 1 rows before, all at once, and its taps, and slides over them in
// registers.  So x is read from memory once (the W - 1 rows again from L2) and y written once: bound by
// memory.  4097 x 8192 bf16 27.2 us from one call to the next (4.9 TB/s), 36.2 with inputs from memory (3.7; a
// copy of as much 26.3), 32768 x 8192 208 (5.2).  Walking down 16 rows with four on their way took 39
// from memory.  Stores that bypass the caches made that 36 and 21 us of 4096 x 4096 15, but what reads q,
// k and v next then waits longer: the convolution and a copy of its outputs 66 us instead of 57.
//
// The first W - 1 tokens of a sequence, whose windows reach into its state, and the new state are one
// thread's work for each sequence and channel group ("heads"); all other rows need nothing but x
// ("tiles").  So a state can be replaced in place, its only reader being its writer, and a single
// token for each sequence is the heads' part alone.
#include "layer_launch.h"

#include <type_traits>

#include "row_device.h"

namespace gdr {

namespace {

constexpr int kThreads = 128;  // 32768 x 8192 208 us, 223 with 256

// How an output's channels go into groups of eight.
enum {
    kWhole,    // without rest
    kOverlap,  // an output's last group begins earlier, so that it is whole: some channels are computed twice
    kPart      // an output has fewer than eight channels: its group goes value by value
};

struct ConvGroups {
    int groups;                           // of eight channels; an output's last one may have fewer
    int first[GDR_CONV_MAX_OUT + 1];      // first group of each output
    int64_t head_blocks, tile_blocks, block0, col_waves;  // col_waves: waves across the channels
};

// A thread's channels: the output, their place in it, and in x; how many there are; and how many of the
// first are another thread's to store.
struct Cols {
    int out, at, channel, n, others;
};
__device__ __forceinline__ Cols cols_of(const ConvArgs& a, const ConvGroups& c, int g) {
    int i = 0;
    while (i + 1 < a.n_out && g >= c.first[i + 1]) ++i;
    const int at = (g - c.first[i]) * 8;
    return Cols{i, at, a.begin[i] + at, a.begin[i + 1] - a.begin[i] - at, 0};
}

// The same with the last group of an output begun earlier.
__device__ __forceinline__ Cols whole_cols_of(const ConvArgs& a, const ConvGroups& c, int g) {
    Cols col = cols_of(a, c, g);
    if (col.n < 8) {
        col.others = 8 - col.n;
        col.at -= col.others, col.channel -= col.others;
    }
    return col;
}

template <bool PART, typename T>
__device__ __forceinline__ void store_own(T* p, const Cols& c, const float (&v)[8]) {
    if (c.others == 0) {
        store8<PART>(p, c.n, v);
    } else {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (i >= c.others) p[i] = rounded(v[i], p);
    }
}

template <typename TW, int W, bool PART>
struct Taps {
    float w[W][8], bias[8];
    __device__ __forceinline__ void load(const ConvArgs& a, const Cols& c) {
        const TW* p = static_cast<const TW*>(a.w) + (int64_t)c.channel * W;
        // the 8 W values of eight channels, in W groups of 8
        float v[W][8];
#pragma unroll
        for (int j = 0; j < W; ++j) load8<PART>(p + 8 * j, c.n * W - 8 * j, v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = v[(i * W + j) / 8][(i * W + j) % 8];
        if (a.bias) {
            load8<PART>(static_cast<const TW*>(a.bias) + c.channel, c.n, bias);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) bias[i] = 0.f;
        }
    }
    // f: the window's W rows, oldest first
    template <typename TX>
    __device__ __forceinline__ void store(const ConvArgs& a, const Cols& c, int64_t row, const float (*f)[8], const TX*) const {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) s = __builtin_fmaf(w[j][i], f[j][i], s);
            y[i] = a.silu ? silu_for(s, static_cast<const TX*>(nullptr)) : s;
        }
        store_own<PART>(static_cast<TX*>(a.out[c.out]) + row * a.out_stride[c.out] + c.at, c, y);
    }
};

// What an overlapping group computes of another thread's channels is not stored: their state may be
// replaced already.
template <typename TX, typename TW, int W, int FORM>
__device__ __forceinline__ void head(const ConvArgs& a, const ConvGroups& c, int64_t item) {
    constexpr bool PART = FORM == kPart;
    if (item >= (int64_t)a.B * c.groups) return;
    const int seq = (int)(item / c.groups);
    const int g = (int)(item % c.groups);
    const Cols col = FORM == kOverlap ? whole_cols_of(a, c, g) : cols_of(a, c, g);
    int64_t first = (int64_t)seq * a.T;
    int len = a.T;
    if (a.cu) {
        const Span s = packed_span(a.cu, seq, a.T);
        first = s.first, len = s.count;
    }
    constexpr int P = W - 1;
    float f[2 * P][8];  // the state's rows, then the sequence's first ones
#pragma unroll
    for (int j = 0; j < P; ++j) {
        if (a.state)
            load8<PART>(static_cast<const TX*>(a.state) + ((int64_t)seq * P + j) * a.D + col.channel, col.n, f[j]);
        else
            for (int i = 0; i < 8; ++i) f[j][i] = 0.f;
        if (j < len)
            load8<PART>(static_cast<const TX*>(a.x) + (first + j) * a.x_stride + col.channel, col.n, f[P + j]);
        else
            for (int i = 0; i < 8; ++i) f[P + j][i] = 0.f;
    }
    if (a.out_state) {
#pragma unroll
        for (int j = 0; j < P; ++j) {  // the last P rows of state and x: row len + j of both
            float v[8];
            if (len >= P) {
                load8<PART>(static_cast<const TX*>(a.x) + (first + len - P + j) * a.x_stride + col.channel, col.n, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = f[j][i];
#pragma unroll
                    for (int l = 1; l < P; ++l)
                        if (len == l) v[i] = f[j + l][i];
                }
            }
            store_own<PART>(static_cast<TX*>(a.out_state) + ((int64_t)seq * P + j) * a.D + col.channel, col, v);
        }
    }
    if (len < 1) return;
    Taps<TW, W, PART> taps;
    taps.load(a, col);
#pragma unroll
    for (int t = 0; t < P; ++t)
        if (t < len) taps.store(a, col, first + t, f + t, static_cast<const TX*>(nullptr));
}

// Which of the tile's rows have their whole window in their own sequence.
template <int W, int TILE>
__device__ __forceinline__ uint64_t whole_windows(const ConvArgs& a, int r0) {
    const int lane = threadIdx.x & 63, r = r0 + lane;
    bool ok = lane < TILE && r < a.rows;
    if (ok && !a.cu) {
        ok = r % a.T >= W - 1;
    } else if (ok) {
        int lo = 0, hi = a.B - 1;  // the last sequence that begins at or before r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        const Span s = packed_span(a.cu, lo, a.T);
        ok = r - s.first >= W - 1 && r - s.first < s.count;
    }
    return __ballot(ok);
}

template <typename TX, typename TW, int W, int TILE, int FORM>
__device__ __forceinline__ void tile(const ConvArgs& a, const ConvGroups& c, int64_t wave) {
    constexpr bool PART = FORM == kPart;
    const int64_t t = wave / c.col_waves;
    const int64_t row0 = t * TILE;
    if (row0 >= a.rows) return;
    const int r0 = (int)row0;
    const uint64_t whole = whole_windows<W, TILE>(a, r0);
    const int g = (int)(wave % c.col_waves) * 64 + (threadIdx.x & 63);
    if (whole == 0 || g >= c.groups) return;
    Cols col = FORM == kOverlap ? whole_cols_of(a, c, g) : cols_of(a, c, g);
    col.others = 0;  // the same values twice: one store for all is quicker
    const TX* x = static_cast<const TX*>(a.x) + col.channel;
    Raw8<TX> raw[W - 1 + TILE];  // all on their way before the first is used
#pragma unroll
    for (int j = 0; j < W - 1 + TILE; ++j) {
        const int r = r0 - (W - 1) + j;
        raw[j] = r >= 0 && r < a.rows ? load8_raw<PART>(x + r * a.x_stride, col.n) : Raw8<TX>{};
    }
    Taps<TW, W, PART> taps;
    taps.load(a, col);
    float f[W - 1 + TILE][8];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j].get(f[j]);
#pragma unroll
    for (int u = 0; u < TILE; ++u) {
        raw[W - 1 + u].get(f[W - 1 + u]);
        if (whole >> u & 1) taps.store(a, col, (int64_t)r0 + u, f + u, static_cast<const TX*>(nullptr));
    }
}

template <typename TX, typename TW, int W, int TILE, int FORM>
__global__ __launch_bounds__(kThreads) void causal_conv_kernel(ConvArgs a, ConvGroups c) {
    const int64_t b = c.block0 + blockIdx.x;
    if (b < c.head_blocks)
        head<TX, TW, W, FORM>(a, c, b * kThreads + threadIdx.x);
    else
        tile<TX, TW, W, TILE, FORM>(a, c, xcd_order(b - c.head_blocks, c.tile_blocks) * (kThreads / 64) +
                                              __builtin_amdgcn_readfirstlane(threadIdx.x / 64));
}

template <typename TX, typename TW, int W>
hipError_t launch(const ConvArgs& a) {
    ConvGroups c{};
    int form = kWhole;
    for (int i = 0; i < a.n_out; ++i) {
        const int n = a.begin[i + 1] - a.begin[i];
        if (n % 8 != 0 && form != kPart) form = n < 8 ? kPart : kOverlap;
        c.first[i] = c.groups;
        c.groups += (n + 7) / 8;
    }
    for (int i = a.n_out; i <= GDR_CONV_MAX_OUT; ++i) c.first[i] = c.groups;
    c.col_waves = (c.groups + 63) / 64;
    c.head_blocks = ((int64_t)a.B * c.groups + kThreads - 1) / kThreads;
    const bool tiles = a.rows > 0 && a.T >= W;  // some sequence may be longer than its head
    auto go = [&](auto rows, auto kernel) {
        constexpr int TILE = decltype(rows)::value;
        const int64_t waves = tiles ? ((int64_t)a.rows + TILE - 1) / TILE * c.col_waves : 0;
        c.tile_blocks = (waves + kThreads / 64 - 1) / (kThreads / 64);
        return by_blocks(c.head_blocks + c.tile_blocks, kThreads, [&](int64_t first, unsigned count) {
            c.block0 = first;
            hipLaunchKernelGGL(kernel, dim3(count), dim3(kThreads), 0, a.stream, a, c);
        });
    };
    // Tiles of 8 rows where they make sixteen waves for each CU, of 4 rows below: more waves count for more
    // than rows read again.  us at 8 / 4 rows, inputs from memory: 32768 x 8192 bf16 208 / 236, 4097 x 8192
    // 36.2 / 38.4, 4097 x 4096 20.4 / 20.2, 3000 x 3000 11.9 / 12.2; 300 x 2048 4.3 at 4, 5.1 at 8.
    using std::integral_constant;
    auto rows = [&](auto n) {
        constexpr int TILE = decltype(n)::value;
        return form == kWhole     ? go(n, causal_conv_kernel<TX, TW, W, TILE, kWhole>)
               : form == kOverlap ? go(n, causal_conv_kernel<TX, TW, W, TILE, kOverlap>)
                                  : go(n, causal_conv_kernel<TX, TW, W, TILE, kPart>);
    };
    return (int64_t)a.rows / 8 * c.col_waves >= 4096 ? rows(integral_constant<int, 8>{}) : rows(integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_causal_conv(const ConvArgs& a) {
    if (a.B < 1 || a.D < 1 || a.n_out < 1 || a.n_out > GDR_CONV_MAX_OUT) return hipErrorInvalidValue;
    auto width = [&](auto x, auto w) {
        using TX = decltype(x);
        using TW = decltype(w);
        return a.W == 2 ? launch<TX, TW, 2>(a) : a.W == 3 ? launch<TX, TW, 3>(a) : a.W == 4 ? launch<TX, TW, 4>(a) : hipErrorInvalidValue;
    };
    if (!a.bf16) return width(float{}, float{});
    return a.w_bf16 ? width(bf16_t{}, bf16_t{}) : width(bf16_t{}, float{});
}

}  // namespace gdr

// Which kernel runs a selective scan, and whether its sequences are cut into segments, by the sizes alone.
#pragma once

#include <stdint.h>

namespace gdr {

// Segments that the sequences of a scan are cut into, by the sizes alone.
//
// A scan runs a token after the other in workgroups of 16 channels: 25 ns a token for one workgroup on a CU, 36,
// 63 and 128 with more than 16, 32 and 64 states.  Where they leave half the CUs idle, segments run side by
// side: first the states behind each from zero, then each segment from its start.  The two launches take the
// time of 125 tokens of a run, and each token of a segment that of 2, or 3.1 with two workgroups on a CU (more
// than 64 states: only one fits, of its registers).  us whole / cut, N = 16: 1 x 511 x 64 15.5 / 9.9, 4097 x 1024 100 / 50,
// 4097 x 2000 100 / 82, 8 x 600 x 256 19.2 / 22.3, 4 x 300 x 256 11.0 / 12.4; N = 32: 4097 x 1024 148 / 74, 3026 x 2592 112 / 122;
// N = 64: 4097 x 1024 258 / 125, 3 x 3496 x 944 224 / 367; N = 128: 4097 x 1024 527 / 285, 8 x 600 x 256 83 / 110.
//
// In a packed batch any sequence may have all rows.  Sequence i, from row c on, has the slots from c / seg_len + i
// on: at least as many as segments, and T / seg_len + B in all, whatever the lengths, which the host does not know.
// Cutting is for lengths that differ; equal ones may lose by it.  us whole / cut, N = 16, equal lengths, and half of the
// rows in one: 10 x 300 x 64 11.6 / 12.3 and 39 / 13.8, 10 x 1200 x 128 33.8 / 30.9 and 141 / 32.3, 20 x 300 x 128 12.4 / 22.8 and
// 72.5 / 23.0, 20 x 600 x 128 22.2 / 33.3 and 142 / 33.2, 40 x 300 x 64 12.8 / 25.3 and 141 / 25.6; N = 128: 20 x 300 x 64 45 / 56 and
// 384 / 77.  Below 512 rows in all both lose, of up to 64 states: 3 x 130 x 64 9.1 / 11.3 and 10.0 / 11.3, N = 64 13.9 / 20.9 and
// 19.5 / 20.9; from there on one of the two wins: 4 x 130 x 64 9.0 / 11.4 and 11.6 / 11.4, 8 x 130 x 64 9.1 / 11.7 and 17.5 / 11.9.
// With more, a run is long enough at once: 2 x 250 x 64, N = 128, 37.9 / 31.1.
struct ScanCut {
    int segs, seg_len;  // packed: segs * B slots
};
inline ScanCut scan_cut(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, bool packed) {
    const int64_t groups = G * ((D / G + 15) / 16), blocks = B * groups;
    const int64_t n = (N > 64 && !packed ? 256 : 512) / blocks, mean = packed ? T / B : T;
    if (n < 3 || mean < (packed ? 128 : 256)) return {1, 0};
    const int64_t len = ((mean + n - 1) / n + 63) / 64 * 64;
    const int64_t segs = packed ? (T / len + 2 * B - 1) / B : (T + len - 1) / len;
    if (segs < 2 || (packed && T < 512 && N <= 64)) return {1, 0};
    if (!packed) {
        const bool two = segs * blocks > 256;
        if ((two && T < 512) || 125 + len * (two ? 31 : 20) / 10 >= T) return {1, 0};
    }
    return {static_cast<int>(segs), static_cast<int>(len)};
}

// Lanes that share a channel in a workgroup of 256 (a channel each 16 or 4 of them), and state values in each.
struct ScanTile {
    int lanes, states;
};

// Tokens of a tile, whose operands lie in LDS twice: two workgroups share a CU's (of more than 64 states one fits by its
// registers, and longer tiles than 16 were not measured).
constexpr int scan_tile_tokens(int lanes, int states) {
    return lanes == 4 ? 32 : states <= 2 ? 64 : states == 4 ? 48 : 16;
}

// Lanes for a channel.  ns a token, by workgroups for each CU (each of the dense batch's sequences as
// long; 256 CUs): 16 lanes, workgroups of 16 channels: 25, 42, 60, 78, 116 for 1, 2, 3, 4, 6; 4 lanes, workgroups
// of 64 channels, N = 16: 74, 135, 270 for 1, 2, 4, N = 8: 103 for 2.  So 4 lanes take less where they
// fill the CUs evenly.  us with 4 lanes / 16: 8 x 512 x 4096 73 / 82, N = 8 55 / 84, 16 x 256 x 4096 77 / 86, 4 x 2048 x 4096 171 / 170;
// 6 x 1024 x 4096 140 / 120, 2 x 2048 x 4096 152 / 94.  Sequences of a packed batch end at different times: there only
// from four workgroups a CU on.
inline bool scan_few_lanes(int64_t B, int64_t D, int64_t N, int64_t G, bool packed, int64_t segs) {
    if (N > 16 || segs > 1) return false;
    const int64_t per = D / G, parts = B * G, wide = parts * ((per + 63) / 64), narrow = parts * ((per + 15) / 16);
    if (packed) return wide >= 1024;
    const int64_t rounds4 = (wide + 255) / 256, rounds16 = (narrow + 255) / 256;
    return rounds4 * (N > 8 ? 67 : 51) < rounds16 * 19;
}

inline ScanTile scan_tile(int64_t B, int64_t D, int64_t N, int64_t G, bool packed, int64_t segs) {
    if (scan_few_lanes(B, D, N, G, packed, segs)) return {4, N <= 8 ? 2 : 4};
    return {16, N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8};
}

}  // namespace gdr

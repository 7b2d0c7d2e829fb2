// int8 matrix product with a scale for each row of a and of w:
//   out[m][n] = (sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
// Sums are int32 in the matrix cores (v_mfma_i32_16x16x64_i8), exact for K <= 131071.  Scales and
// bias are applied in fp32; a bf16 output is rounded once, as it is stored.
//
// Forms, by how many outputs there are (plan() in i8_plan.h): 16 x 16 outputs by 8 waves that share the
// reduction, without LDS staging; small tiles whose waves share the reduction; 128-wide tiles;
// 192 x 256 and 256 x 256 tiles.  At 1 x 12288 x 4096 what is read is the weights: 50 MB in 12.2 us from
// memory, 4.1 TB/s (a large copy reaches 5.1), in 9.9 us from the last-level cache.  At
// 32768 x 4096 x 4096 the chip is limited by power: 447 us, 2460 TOP/s (the library's int8 product
// reaches 2070 on 8192^3).  Times are from one call to the next in a captured graph.
#include "i8_launch.h"

#include <type_traits>

#include "gdr_device.h"
#include "i8_plan.h"

namespace gdr {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// D(16x16, int32) += A(16x64) * B(64x16), int8 operands.  Per lane l: A row l % 16 and B column
// l % 16, 16 consecutive reduction bytes of group l / 16 (the same in both); D rows
// 4 (l / 16) .. + 3 of column l % 16.  A is w and B is a throughout, so that a lane holds four
// consecutive columns of one output row.
__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Bytes at any address.  A load of 16 bytes from an address that is no multiple of 4 is served
// many times slower than one that is (20 x 680 x 3344: 11.7 against 5.7 us), so 16 bytes at p are
// taken from a window of 20 that begins at the multiple of 4 before p, and moved into place.  The
// window is kept inside the operand (`first` to 20 bytes before its end, `last`), so that nothing
// outside it is read; at its two ends the window then begins elsewhere, up to 4 bytes before p.
struct Extent {
    const int8_t *first, *last;
};
__device__ __forceinline__ Extent extent_of(const int8_t* p, int64_t rows, int64_t stride, int K) {
    return Extent{p, p + (rows - 1) * stride + K - 20};
}
struct Window {
    i32x4 v;
    int v4;
    int drop;  // bytes before p, 0 .. 4
};
__device__ __forceinline__ Window load_window(const int8_t* p, Extent e) {
    const int8_t* w = p - (reinterpret_cast<uintptr_t>(p) & 3u);
    w = w < e.first ? e.first : w;
    w = w > e.last ? e.last : w;
    Window r;
    __builtin_memcpy(&r.v, w, 16);
    __builtin_memcpy(&r.v4, w + 16, 4);
    r.drop = (int)(p - w);
    return r;
}
__device__ __forceinline__ i32x4 bytes_of(const Window& w) {
    const bool b = w.drop == 4;
    const uint32_t d[5] = {(uint32_t)(b ? w.v[1] : w.v[0]), (uint32_t)(b ? w.v[2] : w.v[1]), (uint32_t)(b ? w.v[3] : w.v[2]),
                           (uint32_t)(b ? w.v4 : w.v[3]), (uint32_t)w.v4};
    i32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (int)__builtin_amdgcn_alignbyte(d[i + 1], d[i], (uint32_t)w.drop & 3u);
    return r;
}

// v[i] = 16 bytes at p[i] + k[i] of a row of K bytes, zeros from K on.  A chunk that passes the row's
// end is cut from the row's last 16 bytes, so that all loads are under way before one is waited for
// (only rows of fewer than 20 bytes go byte by byte).  e[i]: the operand that p[i] is a row of.
template <int N>
__device__ __forceinline__ void load_cut(const int8_t* const (&p)[N], const int (&k)[N], int K, const Extent (&e)[N],
                                         i32x4 (&v)[N]) {
    if (K >= 20) {
        Window w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = load_window(p[i] + min(k[i], K - 16), e[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const i32x4 u = bytes_of(w[i]);
            const int sh = (k[i] - min(k[i], K - 16)) * 8;  // bits to drop at the low end
            const uint64_t lo = (uint32_t)u[0] | (uint64_t)(uint32_t)u[1] << 32;
            const uint64_t hi = (uint32_t)u[2] | (uint64_t)(uint32_t)u[3] << 32;
            const uint64_t low = sh < 64 ? lo >> (sh & 63) | hi << 1 << (63 - (sh & 63)) : sh < 128 ? hi >> (sh & 63) : 0;
            const uint64_t high = sh < 64 ? hi >> (sh & 63) : 0;
            v[i] = i32x4{(int)low, (int)(low >> 32), (int)high, (int)(high >> 32)};
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (k[i] + j < K) u[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[i][k[i] + j])) << (j % 4 * 8);
            v[i] = i32x4{(int)u[0], (int)u[1], (int)u[2], (int)u[3]};
        }
    }
}

// Where column n goes.
struct Where {
    char* p;  // its address in row 0
    int64_t stride;
    int left;  // columns of the same output from n on
};
__device__ __forceinline__ Where where(const MatmulOut& o, int n, int elt) {
    char* p = static_cast<char*>(o.ptr[0]);
    int64_t stride = o.stride[0];
    int begin = 0, end = o.begin[1];
#pragma unroll
    for (int i = 1; i < GDR_MATMUL_I8_MAX_OUT; ++i)
        if (i < o.n && n >= o.begin[i]) p = static_cast<char*>(o.ptr[i]), stride = o.stride[i], begin = o.begin[i], end = o.begin[i + 1];
    return Where{p + (int64_t)(n - begin) * elt, stride, end - n};
}

template <bool BF16>
__device__ __forceinline__ void store_value(char* p, float x) {
    if constexpr (BF16)
        *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(x);
    else
        *reinterpret_cast<float*>(p) = x;
}

template <bool BF16>
__device__ __forceinline__ void store_bits(char* p, const char* from) {
    if constexpr (BF16)
        *reinterpret_cast<uint16_t*>(p) = *reinterpret_cast<const uint16_t*>(from);
    else
        *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(from);
}

// Columns n .. n+3 of output row m from their sums.
template <bool BF16>
__device__ __forceinline__ void store_quad(const MatmulArgs& g, int m, int n, i32x4 acc) {
    constexpr int E = BF16 ? 2 : 4;
    if (m >= g.M || n >= g.N) return;
    const float sa = g.a_scale[m];
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = min(n + j, g.N - 1);
        v[j] = (float)acc[j] * sa * g.w_scale[c] + (g.bias ? g.bias[c] : 0.f);
    }
    const Where to = where(g.out, n, E);
    if (to.left >= 4) {  // one store, at any alignment
        char* p = to.p + m * to.stride * E;
        if constexpr (BF16) {
            const u32x2 b = bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]});
            __builtin_memcpy(p, &b, 8);
        } else {
            __builtin_memcpy(p, v, 16);
        }
        return;
    }
    // columns of this output, of the next one, and of any after that one by one
    const int all = min(4, g.N - n);
    const Where then = where(g.out, min(n + to.left, g.N - 1), E);
    char *p = to.p + m * to.stride * E, *p2 = then.p + m * then.stride * E;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < min(to.left + then.left, all)) store_value<BF16>(j < to.left ? p + j * E : p2 + (j - to.left) * E, v[j]);
#pragma unroll
    for (int j = 2; j < 4; ++j)
        if (j >= to.left + then.left && j < all) {
            const Where one = where(g.out, n + j, E);
            store_value<BF16>(one.p + m * one.stride * E, v[j]);
        }
}

// Workgroups are dealt to the 8 XCDs in turn; this numbering gives each XCD a run of neighbouring
// tiles, whose shared operands then stay in its L2.
__device__ __forceinline__ int tile_of_workgroup(int total) {
    const int xcd = blockIdx.x & 7, nth = blockIdx.x >> 3;
    return xcd * (total >> 3) + min(xcd, total & 7) + nth;
}

// ---- few outputs ----------------------------------------------------------------------------
// One workgroup makes 16 columns of 16 rows.  Its 8 waves share the reduction, 256 bytes in turn, each
// straight from memory to registers to the matrix cores: every weight is read once and used at
// once, so nothing is gained by LDS; the sums meet there at the end.
// ALIGN: pointers and row strides are multiples of 4 and K is one of 16 (16: chunks are whole), are
// multiples of 4 (4), or anything (1).
template <int ALIGN, bool BF16>
__global__ __launch_bounds__(512) void matmul_rows_kernel(MatmulArgs g) {
    constexpr int WAVES = 8, U = 4, STEP = 64 * U;
    __shared__ i32x4 part[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tiles_m = (g.M + 15) / 16, id = tile_of_workgroup(gridDim.x);
    const int m0 = id % tiles_m * 16, n0 = id / tiles_m * 16, kq = (lane >> 4) * 16;
    const int8_t* pw = g.w + min(n0 + (lane & 15), g.N - 1) * g.w_stride;
    const int8_t* pa = g.a + min(m0 + (lane & 15), g.M - 1) * g.a_stride;
    const Extent ea = extent_of(g.a, g.M, g.a_stride, g.K), ew = extent_of(g.w, g.N, g.w_stride, g.K);
    i32x4 acc = {};
    for (int k0 = wave * STEP; k0 < g.K; k0 += WAVES * STEP) {
        i32x4 fw[U], fa[U];
        if constexpr (ALIGN == 16) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * 64 + kq, from = k < g.K ? k : 0;
                __builtin_memcpy(&fw[u], pw + from, 16);
                __builtin_memcpy(&fa[u], pa + from, 16);
                if (k >= g.K) fw[u] = i32x4{0, 0, 0, 0};
            }
        } else if (ALIGN == 4 && k0 + STEP <= g.K) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                __builtin_memcpy(&fw[u], pw + k0 + u * 64 + kq, 16);
                __builtin_memcpy(&fa[u], pa + k0 + u * 64 + kq, 16);
            }
        } else if (k0 + STEP <= g.K) {
            Window w[U], a[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = load_window(pw + k0 + u * 64 + kq, ew);
                a[u] = load_window(pa + k0 + u * 64 + kq, ea);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) fw[u] = bytes_of(w[u]), fa[u] = bytes_of(a[u]);
        } else {
            const int8_t* p[2 * U];
            int k[2 * U];
            Extent e[2 * U];
            i32x4 v[2 * U];
#pragma unroll
            for (int u = 0; u < 2 * U; ++u) p[u] = u < U ? pw : pa, e[u] = u < U ? ew : ea, k[u] = k0 + u % U * 64 + kq;
            load_cut(p, k, g.K, e, v);
#pragma unroll
            for (int u = 0; u < U; ++u) fw[u] = v[u], fa[u] = v[U + u];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc = mfma_i8(fw[u], fa[u], acc);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        i32x4 s = part[0][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += part[w][lane];
        store_quad<BF16>(g, m0 + (lane & 15), n0 + (lane >> 4) * 4, s);
    }
}

// ---- tiles ------------------------------------------------------------------------------
// One workgroup of WM x WN waves makes BM x BN outputs, 128 reduction bytes at a time through
// STAGES buffers in LDS.  A row's 128 bytes are 8 chunks of 16; chunk c of row r sits at place
// c ^ (r % 8), which spreads the 16 rows that a fragment reads over all banks.
// Operands go from memory to LDS without registers, 16 bytes a lane; a tile's rows lie within 2^31
// bytes.  Copies need addresses that are multiples of 4.  Where rows begin elsewhere (SHIFT) each is
// copied from the aligned word that its first byte lies in, with one more word behind each stage's
// 128 bytes, and a fragment is moved into place, by 0 to 3 bytes, as it is read from LDS.  Words
// are read whole: the first and the last may begin before the operand or end behind it.
// At 4096 x 4096 x K, 256 x 256 tiles, operands from memory: K = 4096 64 us; 4100, where a stage's bytes
// of a row lie in two lines, 80; 4097, moved, 98 (from the last-level cache 54, 63 and 83).  Rows
// moved in registers on their way to LDS took 3 % less there, but 128 x 64 tiles 29 % more.
// What bounds the 256 x 256 form: at 8192^3 the matrix cores are busy 74 % of the time at a clock of
// 1.83 GHz (profiles/int8_product_counters.md); an order of issue with 68 % busy ran at 1.94 GHz and
// took the same time, so it is the power that a product costs.  Tried and dropped (8192^3, against 430 us
// in the same runs): 32x32x32 products, 457;
// four waves of 128 x 128 each, a third fewer LDS reads but nothing to cover a wait, 477; 64-byte
// stages, five deep, 621 (half lines cost as many requests as whole ones); touching lines two
// stages ahead to have them in L2, 515; higher wave priority around the products, 519.
// Rows past the end repeat the last one (their results are dropped); the reduction's last
// partial 128 bytes go through registers, with zeros behind them.
constexpr int kBK = 128;

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
    asm volatile("" ::: "memory");
}

// 16 bytes a lane from r at voff + soff to LDS at `to` + 16 * lane, without registers; one word the
// same way.
typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ void copy_to_lds(rsrc_t r, i32x4* to, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ void copy_word_to_lds(rsrc_t r, int* to, int voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, voff, 0, 0, 0);
}

// The same from an address of each lane's own.
__device__ __forceinline__ void copy_to_lds(const int8_t* from, i32x4* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void*)to, 16, 0, 0);
}
__device__ __forceinline__ void copy_word_to_lds(const int8_t* from, int* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void*)to, 4, 0, 0);
}

// Bytes by .. by + 15 of v and the word behind it.
__device__ __forceinline__ i32x4 moved(i32x4 v, int next, uint32_t by) {
    const uint32_t d[5] = {(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3], (uint32_t)next};
    i32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = (int)__builtin_amdgcn_alignbyte(d[j + 1], d[j], by);
    return r;
}
__device__ __forceinline__ const int8_t* word_of(const int8_t* p) { return p - (reinterpret_cast<uintptr_t>(p) & 3u); }

template <int BM, int BN, int WM, int WN, int STAGES, bool SHIFT, bool BF16>
__global__ __launch_bounds__(WM* WN * 64) void matmul_tile_kernel(MatmulArgs g) {
    constexpr int NT = WM * WN * 64, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int LA = BM * 8 / NT, LW = BN * 8 / NT;
    static_assert(BM * 8 % NT == 0 && BN * 8 % NT == 0 && TM >= 1 && TN >= 1);
    constexpr int ROWS = BM + BN;
    // Stages and, with SHIFT, the word behind each row's 128 bytes.  One array: with several the
    // compiler takes every copy under way to be waited for before any of them is read.
    __shared__ __align__(1024) i32x4 room[STAGES * ROWS * 8 + (SHIFT ? STAGES * ROWS / 4 : 0)];
    i32x4(*const lds)[ROWS * 8] = reinterpret_cast<i32x4(*)[ROWS * 8]>(room);
    int* const words = reinterpret_cast<int*>(room);
    constexpr int BEHIND = STAGES * ROWS * 32;  // words before the words behind
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // an XCD's run of tiles is laid out 8 tiles high, so that those it works on at a time share
    // rows of both operands
    const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
    const int id = tile_of_workgroup(gridDim.x);
    const int band = id / (8 * tiles_n), in_band = id - band * 8 * tiles_n;
    const int high = min(8, tiles_m - band * 8);
    const int m0 = (band * 8 + in_band % high) * BM, n0 = in_band / high * BN;

    const int last_m = min(BM, g.M - m0) - 1, last_n = min(BN, g.N - n0) - 1;
    const int8_t* ga = g.a + m0 * g.a_stride;
    const int8_t* gw = g.w + n0 * g.w_stride;
    // chunk of 16 bytes that this thread brings with its load i: LDS place i * NT + tid
    const int row = tid >> 3, chunk = (tid & 7) ^ (row & 7);
    static_assert(NT % 64 == 0);

    const int full = g.K / kBK;
    // Offsets of this thread's chunks from the first byte of the tile's first row or, with SHIFT,
    // from the word that it lies in.
    const int lead_a = SHIFT ? (int)(reinterpret_cast<uintptr_t>(ga) & 3u) : 0;
    const int lead_w = SHIFT ? (int)(reinterpret_cast<uintptr_t>(gw) & 3u) : 0;
    const int bytes_a = lead_a + last_m * (int)g.a_stride + g.K, bytes_w = lead_w + last_n * (int)g.w_stride + g.K;
    const rsrc_t ra = make_rsrc(ga - lead_a, SHIFT ? (uint32_t)(bytes_a + 3) & ~3u : (uint32_t)bytes_a);
    const rsrc_t rw = make_rsrc(gw - lead_w, SHIFT ? (uint32_t)(bytes_w + 3) & ~3u : (uint32_t)bytes_w);
    auto start_a = [&](int r) {
        const int at = min(r, last_m) * (int)g.a_stride + lead_a;
        return SHIFT ? at & ~3 : at;
    };
    auto start_w = [&](int r) {
        const int at = min(r, last_n) * (int)g.w_stride + lead_w;
        return SHIFT ? at & ~3 : at;
    };
    int va[LA], vw[LW];
#pragma unroll
    for (int i = 0; i < LA; ++i) va[i] = start_a(row + i * (NT / 8)) + chunk * 16;
#pragma unroll
    for (int i = 0; i < LW; ++i) vw[i] = start_w(row + i * (NT / 8)) + chunk * 16;
    // Each wave copies the words behind 64 rows.  A word past the operand's last one would belong
    // to a row that begins at a whole word, which needs none: the last one is read in its place.
    static_assert(!SHIFT || (BM % 64 == 0 && BN % 64 == 0 && ROWS / 64 <= WM * WN));
    const int group = wave % (ROWS / 64) * 64;
    const bool group_a = group < BM;
    const int vb = group_a ? start_a(group + lane) : start_w(group - BM + lane);
    const int last_word = ((group_a ? bytes_a : bytes_w) - 1) & ~3;
    constexpr int L = LA + LW + (SHIFT ? 1 : 0);  // copies of a stage
    const Extent ea = extent_of(g.a, g.M, g.a_stride, g.K), ew = extent_of(g.w, g.N, g.w_stride, g.K);
    auto fetch = [&](int s) {
        const int k = s * kBK;
        i32x4* to = &lds[s % STAGES][wave * 64];
#pragma unroll
        for (int i = 0; i < LA; ++i) copy_to_lds(ra, to + i * NT, va[i], k);
#pragma unroll
        for (int i = 0; i < LW; ++i) copy_to_lds(rw, to + BM * 8 + i * NT, vw[i], k);
        if constexpr (SHIFT) {
            int* word = &words[BEHIND + s % STAGES * ROWS + group];
            const int v = min(vb + k + kBK, last_word);
            if (group_a)
                copy_word_to_lds(ra, word, v);
            else
                copy_word_to_lds(rw, word, v);
        }
    };

    i32x4 acc[TM][TN] = {};
    const int wm = wave / WN, wn = wave % WN;
    // place of this lane's chunk of a fragment: row lane % 16, chunk lane / 16 (+ 4 for the second
    // half of the 128 bytes)
    const int place = (lane & 15) * 8 + ((lane >> 4) ^ (lane & 7));
    struct Frags {
        i32x4 a[TM], w[TN];
    };
    auto read = [&](int s, int h, Frags& f) {
        const i32x4* A = &lds[s % STAGES][wm * (TM * 128)];
        const i32x4* W = &lds[s % STAGES][BM * 8 + wn * (TN * 128)];
#pragma unroll
        for (int j = 0; j < TN; ++j) f.w[j] = W[j * 128 + (place ^ (h * 4))];
#pragma unroll
        for (int i = 0; i < TM; ++i) f.a[i] = A[i * 128 + (place ^ (h * 4))];
    };
    // The same, moved into place.  Rows 16 apart begin alike in a word (those past the end may not;
    // their results are dropped).  Behind chunk 7 is the word from `behind`.
    const int quarter = lane >> 4;
    const uint32_t by_a = ((uint32_t)lead_a + (uint32_t)(wm * TM * 16 + (lane & 15)) * (uint32_t)g.a_stride) & 3u;
    const uint32_t by_w = ((uint32_t)lead_w + (uint32_t)(wn * TN * 16 + (lane & 15)) * (uint32_t)g.w_stride) & 3u;
    const bool past = quarter == 3;  // in a stage's second half
    const int next0 = (lane & 15) * 32 + ((quarter + 1) ^ (lane & 7)) * 4;
    const int next1 = past ? BEHIND + wm * (TM * 16) + (lane & 15) : wm * (TM * 512) + (lane & 15) * 32 + ((quarter + 5) ^ (lane & 7)) * 4;
    const int next2 = past ? BEHIND + BM + wn * (TN * 16) + (lane & 15)
                           : BM * 32 + wn * (TN * 512) + (lane & 15) * 32 + ((quarter + 5) ^ (lane & 7)) * 4;
    const int apart1 = past ? 16 : 512, stage1 = past ? ROWS : ROWS * 32;
    auto read_moved = [&](int s, int h, Frags& f) {
        const int b = s % STAGES;
        read(s, h, f);
        const int* A = words + (h ? next1 + b * stage1 : b * (ROWS * 32) + wm * (TM * 512) + next0);
        const int* W = words + (h ? next2 + b * stage1 : b * (ROWS * 32) + BM * 32 + wn * (TN * 512) + next0);
        const int apart = h ? apart1 : 512;
        int na[TM], nw[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) nw[j] = W[j * apart];
#pragma unroll
        for (int i = 0; i < TM; ++i) na[i] = A[i * apart];
#pragma unroll
        for (int j = 0; j < TN; ++j) f.w[j] = moved(f.w[j], nw[j], by_w);
#pragma unroll
        for (int i = 0; i < TM; ++i) f.a[i] = moved(f.a[i], na[i], by_a);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma_i8(f.w[j], f.a[i], acc[i][j]);
    };
    auto compute = [&](int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Frags f;
            read(s, h, f);
            multiply(f);
        }
    };

#pragma unroll
    for (int s = 0; s < STAGES; ++s)
        if (s < full) fetch(s);
    if (full >= STAGES)
        wait_vmcnt<(STAGES - 1) * L>();
    else
        wait_vmcnt<0>();
    lds_barrier();
    if constexpr (!SHIFT) {
        // Two sets of fragments: while one half of a stage is multiplied the next half is read
        // from LDS, also across stages: the barrier that frees stage s (everyone has read it) and
        // opens stage s + 1 stands between the halves of stage s.  The order is written out, a
        // row of products at a time: LDS reads go with the first rows (two each, so that the last
        // are back before the next half needs them), copies to LDS one or two with each row, since
        // a run of copies holds a wave up while the address unit takes 64 lanes' worth each.
        constexpr int RD = TM + TN, PR = (RD + TM - 1) / TM + 1, PL = (L + TM - 1) / TM;
        Frags f0, f1;
        auto half = [&](const Frags& use, Frags& next, int rs, int rh, auto reads, int fs, auto copies) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if constexpr (decltype(reads)::value) {
#pragma unroll
                    for (int r = i * PR; r < (i + 1) * PR && r < RD; ++r) {
                        if (r < TN)
                            next.w[r] = lds[rs % STAGES][BM * 8 + wn * (TN * 128) + r * 128 + (place ^ (rh * 4))];
                        else
                            next.a[r - TN] = lds[rs % STAGES][wm * (TM * 128) + (r - TN) * 128 + (place ^ (rh * 4))];
                    }
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma_i8(use.w[j], use.a[i], acc[i][j]);
                if constexpr (decltype(copies)::value) {
#pragma unroll
                    for (int c = i * PL; c < (i + 1) * PL && c < L; ++c) {
                        i32x4* to = &lds[fs % STAGES][wave * 64];
                        if (c < LA)
                            copy_to_lds(ra, to + c * NT, va[c], fs * kBK);
                        else
                            copy_to_lds(rw, to + BM * 8 + (c - LA) * NT, vw[c - LA], fs * kBK);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto step = [&](int s, auto more, auto next) {
            half(f0, f1, s, 1, std::true_type{}, 0, std::false_type{});
            if constexpr (decltype(next)::value) {
                if constexpr (decltype(more)::value)
                    wait_vmcnt<(STAGES - 2) * L>();
                else
                    wait_vmcnt<0>();
                lds_barrier();
            }
            half(f1, f0, s + 1, 0, next, s + STAGES, more);
        };
        using yes = std::true_type;
        using no = std::false_type;
        if (full > 0) {
            read(0, 0, f0);
            int s = 0;
            for (; s + STAGES < full; ++s) step(s, yes{}, yes{});
            for (; s + 1 < full; ++s) step(s, no{}, yes{});
            step(s, no{}, no{});
        }
    } else {
        // One set: the barrier that frees stage s and opens the next stands where all of its
        // fragments have been read and half of them are multiplied.
        for (int s = 0; s < full; ++s) {
            Frags f;
            read_moved(s, 0, f);
            multiply(f);
            read_moved(s, 1, f);
            if (s + 1 < full) {
                if (s + STAGES - 1 < full)
                    wait_vmcnt<(STAGES - 2) * L>();
                else
                    wait_vmcnt<0>();
                lds_barrier();
                if (s + STAGES < full) fetch(s + STAGES);
            }
            multiply(f);
        }
    }
    if (g.K % kBK != 0) {
        const int s = full;
        const int8_t* p[LA + LW];
        int k[LA + LW];
        Extent e[LA + LW];
        i32x4 v[LA + LW];
#pragma unroll
        for (int i = 0; i < LA + LW; ++i) {
            k[i] = full * kBK + chunk * 16;
            e[i] = i < LA ? ea : ew;
            p[i] = i < LA ? ga + min(row + i * (NT / 8), last_m) * g.a_stride
                          : gw + min(row + (i - LA) * (NT / 8), last_n) * g.w_stride;
        }
        load_cut(p, k, g.K, e, v);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LA + LW; ++i) lds[s % STAGES][(i < LA ? i * NT : BM * 8 + (i - LA) * NT) + tid] = v[i];
        __syncthreads();
        compute(s);
    }

    // Outputs leave through LDS, each wave's block for itself, so that stores are whole lines: a
    // lane's accumulators are four columns of each of TM rows, 32 bytes of a line at a time (stored
    // straight, a 256 x 256 tile took 15 us longer).  Chunk c of 16 bytes of row r sits at place
    // c ^ (r % CH).
    constexpr int E = BF16 ? 2 : 4, CW = TN * 16, EB = CW * E, CH = EB / 16, PER = 16 / E;
    constexpr int SPACE = STAGES * (BM + BN) * kBK / (WM * WN), RP = SPACE / EB < TM * 16 ? SPACE / EB / 16 * 16 : TM * 16;
    static_assert(RP >= 16 && TM * 16 % RP == 0 && CW <= 64);
    float sa[TM];
    f32x4 sw[TN], bias[TN];
    const int mw = m0 + wm * (TM * 16), nw = n0 + wn * CW;
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = g.a_scale[min(mw + i * 16 + (lane & 15), g.M - 1)];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int n = min(nw + j * 16 + (lane >> 4) * 4 + c, g.N - 1);
            sw[j][c] = g.w_scale[n];
            bias[j][c] = g.bias ? g.bias[n] : 0.f;
        }
    const int col = lane % CH * PER, first = lane / CH;  // 16 bytes of columns and the first row of this lane's stores
    constexpr int step_r = 64 / CH;
    const bool on = nw + col < g.N;
    // they go to one output or two; columns from `both` on, of a third one and more, one by one
    const Where to = where(g.out, min(nw + col, g.N - 1), E);
    const int own = min(to.left, PER), all = min(PER, g.N - nw - col);
    Where then = to;
    if (own < all) then = where(g.out, nw + col + own, E);
    const int both = min(own + then.left, all);
    char* mine = reinterpret_cast<char*>(&lds[0][0]) + wave * SPACE;
    lds_barrier();
#pragma unroll
    for (int pass = 0; pass < TM * 16 / RP; ++pass) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < RP / 16; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int t = pass * (RP / 16) + i, r = i * 16 + (lane & 15), q = lane >> 4;
                f32x4 v;
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = (float)acc[t][j][c] * sa[t] * sw[j][c] + bias[j][c];
                const int c16 = BF16 ? j * 2 + (q >> 1) : j * 4 + q;
                char* at = mine + r * EB + (c16 ^ (r & (CH - 1))) * 16;
                if constexpr (BF16) {
                    const u32x2 b = bf16x4_bits(v);
                    __builtin_memcpy(__builtin_assume_aligned(at + (q & 1) * 8, 8), &b, 8);
                } else {
                    __builtin_memcpy(__builtin_assume_aligned(at, 16), &v, 16);
                }
            }
        asm volatile("" ::: "memory");
        const int rows = min(RP, g.M - mw - pass * RP);
        if (!on) continue;
        char* p = to.p + (int64_t)(mw + pass * RP + first) * to.stride * E;
        for (int r = first; r < rows; r += step_r, p += step_r * to.stride * E) {
            const char* at = mine + r * EB + (col / PER ^ (r & (CH - 1))) * 16;
            if (to.left >= PER) {  // one store, at any alignment
                u32x4 x;
                __builtin_memcpy(&x, __builtin_assume_aligned(at, 16), 16);
                __builtin_memcpy(p, &x, 16);
            } else {
                const int64_t m = mw + pass * RP + r;
                char* p2 = then.p + m * then.stride * E;
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    if (c < both) store_bits<BF16>(c < own ? p + c * E : p2 + (c - own) * E, at + c * E);
#pragma unroll 1
                for (int c = both; c < all; ++c) {
                    const Where one = where(g.out, nw + col + c, E);
                    store_bits<BF16>(one.p + m * one.stride * E, at + c * E);
                }
            }
        }
    }
}

// ---- small tiles --------------------------------------------------------------------------
// For products whose larger tiles would leave most of the chip idle.  BM x BN outputs for a
// workgroup; each wave makes a 32 x 32 block, and KG groups of waves share the reduction: a stage
// is KG * 64 bytes of it, group k takes the k-th 64, and the groups' sums meet in LDS.  What bounds
// these products is how fast a CU can bring its operands in, so the loop keeps STAGES - 1 stages
// in flight.  32 x 12288 x 4096: 15.4 us with the weights from memory, 3.3 TB/s, 11.0 from the last-level
// cache; 128 x 4096 x 4096: 11.4 and 8.7 us, where each CU brings 393 KB in at 34 and 45 bytes a ns.
template <int BM, int BN, int KG, int STAGES, bool SHIFT, bool BF16>
__global__ __launch_bounds__(BM / 32 * (BN / 32) * KG * 64) void matmul_small_kernel(MatmulArgs g) {
    constexpr int WN = BN / 32, WAVES = BM / 32 * WN * KG, NT = WAVES * 64;
    constexpr int BK = KG * 64, CPR = BK / 16, ROWS = BM + BN, LD = ROWS * CPR / NT;
    static_assert(KG >= 2 && ROWS * CPR % NT == 0 && NT % CPR == 0);
    constexpr int RED = KG * BM * BN / 4;  // 16-byte places
    constexpr int GROUPS = (ROWS + 63) / 64, L = LD + (SHIFT ? 1 : 0);
    constexpr int STAGED = STAGES * ROWS * CPR + (SHIFT ? STAGES * GROUPS * 16 : 0);
    __shared__ __align__(1024) i32x4 lds[STAGED > RED ? STAGED : RED];
    int* const words = reinterpret_cast<int*>(lds);
    constexpr int BEHIND = STAGES * ROWS * CPR * 4;  // the words behind each row's BK bytes
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // an XCD's tiles share columns of w, the larger operand in these products
    const int tiles_m = (g.M + BM - 1) / BM;
    const int id = tile_of_workgroup(gridDim.x);
    const int m0 = id % tiles_m * BM, n0 = id / tiles_m * BN;
    const int last_m = min(BM, g.M - m0) - 1, last_n = min(BN, g.N - n0) - 1;
    const int8_t* ga = g.a + m0 * g.a_stride;
    const int8_t* gw = g.w + n0 * g.w_stride;

    // A row's CPR chunks of 16 bytes: chunk c of row r sits at place c ^ (r % 8) (CPR >= 8).
    const int row = tid / CPR, chunk = (tid % CPR) ^ (row & 7);
    static_assert(NT / CPR % 8 == 0, "rows of one thread's loads agree modulo 8");
    const int full = g.K / BK;
    const Extent ea = extent_of(g.a, g.M, g.a_stride, g.K), ew = extent_of(g.w, g.N, g.w_stride, g.K);
    auto extent = [&](int i) { return row + i * (NT / CPR) < BM ? ea : ew; };
    auto source = [&](int i) {  // start of the row that this thread's load i brings a chunk of
        const int r = row + i * (NT / CPR);
        return r < BM ? ga + min(r, last_m) * g.a_stride : gw + min(r - BM, last_n) * g.w_stride;
    };
    const int8_t* src[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) src[i] = (SHIFT ? word_of(source(i)) : source(i)) + chunk * 16;
    // each wave copies the words behind 64 rows (as in the tile kernel)
    static_assert(GROUPS <= WAVES);
    const int group = wave % GROUPS * 64, brow = min(group + lane, ROWS - 1);
    const bool in_a = brow < BM;
    const int8_t* bsrc = word_of(in_a ? ga + min(brow, last_m) * g.a_stride : gw + min(brow - BM, last_n) * g.w_stride);
    const int8_t* blast = word_of(in_a ? ga + last_m * g.a_stride + g.K - 1 : gw + last_n * g.w_stride + g.K - 1);

    i32x4 rest[LD];  // the last partial stage
    const bool partial = g.K % BK != 0;
    if (partial) {
        const int8_t* p[LD];
        int k[LD];
        Extent e[LD];
#pragma unroll
        for (int i = 0; i < LD; ++i) p[i] = source(i), k[i] = full * BK + chunk * 16, e[i] = extent(i);
        load_cut(p, k, g.K, e, rest);
    }
    i32x4 acc[2][2] = {};
    const int kg = wave % KG, block = wave / KG, wm = block / WN, wn = block % WN;
    const int place = (lane & 15) * CPR + ((kg * 4 + (lane >> 4)) ^ (lane & 7));
    const int quarter = kg * 4 + (lane >> 4);  // this lane's chunk
    const uint32_t by_a = (uint32_t)(reinterpret_cast<uintptr_t>(ga) + (wm * 32 + (lane & 15)) * g.a_stride) & 3u;
    const uint32_t by_w = (uint32_t)(reinterpret_cast<uintptr_t>(gw) + (wn * 32 + (lane & 15)) * g.w_stride) & 3u;
    auto compute = [&](int buf, auto move) {
        const i32x4* A = &lds[buf * ROWS * CPR + wm * 32 * CPR];
        const i32x4* W = &lds[buf * ROWS * CPR + (BM + wn * 32) * CPR];
        i32x4 fa[2], fw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) fw[i] = W[i * 16 * CPR + place], fa[i] = A[i * 16 * CPR + place];
        if constexpr (decltype(move)::value) {
            const bool past = quarter == CPR - 1;
            const int next = (buf * ROWS * CPR + (lane & 15) * CPR + ((quarter + 1) ^ (lane & 7))) * 4;
            const int behind = BEHIND + buf * GROUPS * 64 + (lane & 15), apart = past ? 16 : 16 * CPR * 4;
            const int* nA = words + (past ? behind + wm * 32 : next + wm * 32 * CPR * 4);
            const int* nW = words + (past ? behind + BM + wn * 32 : next + (BM + wn * 32) * CPR * 4);
            const int n[4] = {nA[0], nA[apart], nW[0], nW[apart]};
#pragma unroll
            for (int i = 0; i < 2; ++i) fa[i] = moved(fa[i], n[i], by_a), fw[i] = moved(fw[i], n[2 + i], by_w);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma_i8(fw[j], fa[i], acc[i][j]);
    };
    auto fetch = [&](int s, int buf) {
#pragma unroll
        for (int i = 0; i < LD; ++i) copy_to_lds(src[i] + s * BK, &lds[buf * ROWS * CPR + i * NT + wave * 64]);
        if constexpr (SHIFT) {
            const int8_t* from = bsrc + (s + 1) * BK;
            copy_word_to_lds(from < blast ? from : blast, &words[BEHIND + buf * GROUPS * 64 + group]);
        }
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < full) fetch(s, s);
    int buf = 0;
    for (int s = 0; s < full; ++s) {
        if (s + STAGES - 2 < full)
            wait_vmcnt<(STAGES - 2) * L>();
        else
            wait_vmcnt<0>();
        lds_barrier();
        if (s + STAGES - 1 < full) fetch(s + STAGES - 1, buf == 0 ? STAGES - 1 : buf - 1);
        compute(buf, std::integral_constant<bool, SHIFT>{});
        buf = buf + 1 == STAGES ? 0 : buf + 1;
    }
    if (partial) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LD; ++i) lds[i * NT + tid] = rest[i];
        __syncthreads();
        compute(0, std::false_type{});
    }

    // Sums of the groups meet in LDS: BM x BN int32 each, a row's places of 4 columns exchanged by
    // its number.
    __syncthreads();
    constexpr int QR = BN / 4;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = wm * 32 + i * 16 + (lane & 15), q = wn * 8 + j * 4 + (lane >> 4);
            lds[kg * BM * QR + r * QR + (q ^ (r & 7))] = acc[i][j];
        }
    __syncthreads();
    for (int e = tid; e < BM * QR; e += NT) {
        const int r = e / QR, q = e % QR;
        i32x4 sum = lds[r * QR + (q ^ (r & 7))];
#pragma unroll
        for (int k = 1; k < KG; ++k) sum += lds[k * BM * QR + r * QR + (q ^ (r & 7))];
        store_quad<BF16>(g, m0 + r, n0 + q * 4, sum);
    }
}

template <int ALIGN>
void rows(const MatmulArgs& g) {
    const dim3 grid((unsigned)(((int64_t)g.M + 15) / 16 * ((g.N + 15) / 16)));
    if (g.out_bf16)
        hipLaunchKernelGGL((matmul_rows_kernel<ALIGN, true>), grid, dim3(512), 0, g.stream, g);
    else
        hipLaunchKernelGGL((matmul_rows_kernel<ALIGN, false>), grid, dim3(512), 0, g.stream, g);
}

template <int BM, int BN, int KG, int STAGES, bool SHIFT>
void small(const MatmulArgs& g) {
    const dim3 grid((unsigned)(((int64_t)g.M + BM - 1) / BM * ((g.N + BN - 1) / BN)));
    constexpr int NT = BM / 32 * (BN / 32) * KG * 64;
    if (g.out_bf16)
        hipLaunchKernelGGL((matmul_small_kernel<BM, BN, KG, STAGES, SHIFT, true>), grid, dim3(NT), 0, g.stream, g);
    else
        hipLaunchKernelGGL((matmul_small_kernel<BM, BN, KG, STAGES, SHIFT, false>), grid, dim3(NT), 0, g.stream, g);
}

template <int BM, int BN, int WM, int WN, int STAGES, bool SHIFT>
void tiles(const MatmulArgs& g) {
    const dim3 grid((unsigned)(((int64_t)g.M + BM - 1) / BM * ((g.N + BN - 1) / BN)));
    if (g.out_bf16)
        hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, STAGES, SHIFT, true>), grid, dim3(WM * WN * 64), 0, g.stream, g);
    else
        hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, STAGES, SHIFT, false>), grid, dim3(WM * WN * 64), 0, g.stream, g);
}

template <bool SHIFT>
void start(Form f, const MatmulArgs& g) {
    switch (f) {
        case Form::rows: SHIFT ? rows<1>(g) : g.K % 16 == 0 ? rows<16>(g) : rows<4>(g); break;
        case Form::t32x32: small<32, 32, 8, 3, SHIFT>(g); break;
        case Form::t32x64: small<32, 64, 4, 3, SHIFT>(g); break;
        case Form::t128x64: tiles<128, 64, 4, 2, 3, SHIFT>(g); break;
        case Form::t128x128_deep: tiles<128, 128, 2, 4, 4, false>(g); break;  // of whole words only
        case Form::t128x128: tiles<128, 128, 2, 4, 2, SHIFT>(g); break;
        case Form::t192x256: tiles<192, 256, 2, 4, 2, SHIFT>(g); break;
        case Form::t256x256: tiles<256, 256, 2, 4, 2, SHIFT>(g); break;
    }
}

MatmulArgs rows_of(const MatmulArgs& g, int first, int count) {
    MatmulArgs r = g;
    r.M = count;
    r.a += first * g.a_stride;
    r.a_scale += first;
    for (int i = 0; i < g.out.n; ++i)
        r.out.ptr[i] = static_cast<char*>(g.out.ptr[i]) + first * g.out.stride[i] * (g.out_bf16 ? 2 : 4);
    return r;
}

hipError_t launch(Form f, bool moved, const MatmulArgs& g) {
    moved ? start<true>(f, g) : start<false>(f, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_i8(const MatmulArgs& g) {
    if (g.M < 1 || g.M > GDR_I8_MAX_ROWS || g.N < 1 || g.K < 1 || g.K > GDR_MATMUL_I8_MAX_K) return hipErrorInvalidValue;
    hipError_t e = hipErrorInvalidValue;
    const Operands all{reinterpret_cast<uintptr_t>(g.a), reinterpret_cast<uintptr_t>(g.w), g.M, g.N, g.K, g.a_stride, g.w_stride};
    launches(all, 0, [&](int first, int count, Form form, bool moved) {
        e = launch(form, moved, rows_of(g, first, count));
        return e == hipSuccess;
    });
    return e;
}

}  // namespace gdr

// int8 matrix product with a scale for each row of a and of w:
//   out[m][n] = (sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
// Sums are int32 in the matrix cores (v_mfma_i32_16x16x64_i8), exact for K <= 131071.  Scales and
// bias are applied in fp32; a bf16 output is rounded once, as it is stored.
//
// Forms, by how many outputs there are (see plan()): 16 x 16 outputs by 8 waves that share the
// reduction, without LDS staging; small tiles whose waves share the reduction; 128-wide tiles;
// 256 x 256 tiles.  At 1 x 12288 x 4096 what is read is the weights: 50 MB in 10.4 us, 4.8 TB/s,
// the rate of a large copy being 5.1.  At 32768 x 4096 x 4096 the chip is limited by power: 447 us,
// 2460 TOP/s (the library's int8 product reaches 2070 on 8192^3).
#include "i8_launch.h"

#include <algorithm>
#include <type_traits>

#include "gdr_device.h"

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

// Where the outputs of columns n .. n+3 go: for each column its output's first value of row 0
// and the distance between rows.  Columns of one output share both.
struct Where {
    char* p;  // address of column n in row 0
    int64_t stride;
};
__device__ __forceinline__ Where where(const MatmulOut& o, int n, int elt) {
    char* p = static_cast<char*>(o.ptr[0]);
    int64_t stride = o.stride[0];
    int begin = 0;
#pragma unroll
    for (int i = 1; i < GDR_MATMUL_I8_MAX_OUT; ++i)
        if (i < o.n && n >= o.begin[i]) p = static_cast<char*>(o.ptr[i]), stride = o.stride[i], begin = o.begin[i];
    return Where{p + (int64_t)(n - begin) * elt, stride};
}

template <bool BF16>
__device__ __forceinline__ void store_value(char* p, float x) {
    if constexpr (BF16)
        *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(x);
    else
        *reinterpret_cast<float*>(p) = x;
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
    if (g.out.quad && n + 4 <= g.N) {
        const Where to = where(g.out, n, E);
        char* p = to.p + m * to.stride * E;
        if constexpr (BF16)
            *reinterpret_cast<u32x2*>(p) = bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]});
        else
            *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < g.N) {
            const Where to = where(g.out, n + j, E);
            store_value<BF16>(to.p + m * to.stride * E, v[j]);
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
//   DMA   memory to LDS without registers (16 bytes a lane): pointers and row strides are
//         multiples of 16 and a tile's rows lie within 2^31 bytes;
//   else  through registers, at any alignment, a stage ahead.
// What bounds the 256 x 256 form: at 8192^3 the matrix cores are busy 74 % of the time at a clock of
// 1.83 GHz; an order of issue with 68 % busy ran at 1.94 GHz and took the same time, so it is the
// power that a product costs.  Tried and dropped (8192^3, 430 us): 32x32x32 products, 457;
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

// 16 bytes a lane from r at voff + soff to LDS at `to` + 16 * lane, without registers.
typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ void copy_to_lds(rsrc_t r, i32x4* to, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, voff, soff, 0, 0);
}

// The same from an address of each lane's own.
__device__ __forceinline__ void copy_to_lds(const int8_t* from, i32x4* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void*)to, 16, 0, 0);
}

template <int BM, int BN, int WM, int WN, int STAGES, bool DMA, bool BF16>
__global__ __launch_bounds__(WM* WN * 64) void matmul_tile_kernel(MatmulArgs g) {
    constexpr int NT = WM * WN * 64, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int LA = BM * 8 / NT, LW = BN * 8 / NT;
    static_assert(BM * 8 % NT == 0 && BN * 8 % NT == 0 && TM >= 1 && TN >= 1);
    __shared__ __align__(1024) i32x4 lds[STAGES][(BM + BN) * 8];
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
    int va[LA], vw[LW];
    rsrc_t ra, rw;
    if constexpr (DMA) {
        ra = make_rsrc(ga, (uint32_t)(last_m * g.a_stride + g.K));
        rw = make_rsrc(gw, (uint32_t)(last_n * g.w_stride + g.K));
#pragma unroll
        for (int i = 0; i < LA; ++i) va[i] = min(row + i * (NT / 8), last_m) * (int)g.a_stride + chunk * 16;
#pragma unroll
        for (int i = 0; i < LW; ++i) vw[i] = min(row + i * (NT / 8), last_n) * (int)g.w_stride + chunk * 16;
    }
    const Extent ea = extent_of(g.a, g.M, g.a_stride, g.K), ew = extent_of(g.w, g.N, g.w_stride, g.K);
    i32x4 hold[DMA ? 1 : LA + LW];
    auto fetch = [&](int s) {
        const int k = s * kBK;
        if constexpr (DMA) {
            i32x4* to = &lds[s % STAGES][wave * 64];
#pragma unroll
            for (int i = 0; i < LA; ++i) copy_to_lds(ra, to + i * NT, va[i], k);
#pragma unroll
            for (int i = 0; i < LW; ++i) copy_to_lds(rw, to + BM * 8 + i * NT, vw[i], k);
        } else {
#pragma unroll
            for (int i = 0; i < LA; ++i)
                __builtin_memcpy(&hold[i], ga + min(row + i * (NT / 8), last_m) * g.a_stride + (k + chunk * 16), 16);
#pragma unroll
            for (int i = 0; i < LW; ++i)
                __builtin_memcpy(&hold[LA + i], gw + min(row + i * (NT / 8), last_n) * g.w_stride + (k + chunk * 16), 16);
        }
    };
    auto put = [&](int s) {
        if constexpr (!DMA) {
#pragma unroll
            for (int i = 0; i < LA; ++i) lds[s % STAGES][i * NT + tid] = hold[i];
#pragma unroll
            for (int i = 0; i < LW; ++i) lds[s % STAGES][BM * 8 + i * NT + tid] = hold[LA + i];
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

    if constexpr (DMA) {
        // Two sets of fragments: while one half of a stage is multiplied the next half is read
        // from LDS, also across stages: the barrier that frees stage s (everyone has read it) and
        // opens stage s + 1 stands between the halves of stage s.  The order is written out, a
        // row of products at a time: LDS reads go with the first rows (two each, so that the last
        // are back before the next half needs them), copies to LDS one or two with each row, since
        // a run of copies holds a wave up while the address unit takes 64 lanes' worth each.
        constexpr int L = LA + LW, RD = TM + TN, PR = (RD + TM - 1) / TM + 1, PL = (L + TM - 1) / TM;
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
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (s < full) fetch(s);
        if (full >= STAGES)
            wait_vmcnt<(STAGES - 1) * L>();
        else
            wait_vmcnt<0>();
        lds_barrier();
        if (full > 0) {
            read(0, 0, f0);
            int s = 0;
            for (; s + STAGES < full; ++s) step(s, yes{}, yes{});
            for (; s + 1 < full; ++s) step(s, no{}, yes{});
            step(s, no{}, no{});
        }
    } else {
        if (full > 0) {
            fetch(0);
            put(0);
        }
        for (int s = 0; s < full; ++s) {
            lds_barrier();
            if (s + 1 < full) fetch(s + 1);
            compute(s);
            if (s + 1 < full) put(s + 1);
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
    const bool wide = g.out.wide;
    const int col = wide ? lane % CH * PER : lane % CW;          // of this lane's stores
    const int first = wide ? lane / CH : lane / CW;              // and its first row
    const int step_r = wide ? 64 / CH : 64 / CW;
    const bool on = nw + col < g.N;
    const Where to = where(g.out, min(nw + col, g.N - 1), E);
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
            if (wide) {
                u32x4 x;
                __builtin_memcpy(&x, __builtin_assume_aligned(at, 16), 16);
                *reinterpret_cast<u32x4*>(p) = x;
            } else if constexpr (BF16) {
                uint16_t x;
                __builtin_memcpy(&x, __builtin_assume_aligned(at + col % PER * E, 2), 2);
                *reinterpret_cast<uint16_t*>(p) = x;
            } else {
                float x;
                __builtin_memcpy(&x, __builtin_assume_aligned(at + col % PER * E, 4), 4);
                *reinterpret_cast<float*>(p) = x;
            }
        }
    }
}

// ---- small tiles --------------------------------------------------------------------------
// For products whose 256 x 256 tiles would leave most of the chip idle.  BM x BN outputs for a
// workgroup; each wave makes a 32 x 32 block, and KG groups of waves share the reduction: a stage
// is KG * 64 bytes of it, group k takes the k-th 64, and the groups' sums meet in LDS.  What bounds
// these products is how fast a CU can bring its operands in, so the loop keeps STAGES - 1 stages
// in flight (DMA), or REGS stages in registers (any alignment).  32 x 12288 x 4096: 10.7 us, 4.8
// TB/s; 128 x 4096 x 4096: 9.7 us, where each CU brings 393 KB in at 50 bytes a ns.
template <int BM, int BN, int KG, int STAGES, int REGS, bool DMA, bool BF16>
__global__ __launch_bounds__(BM / 32 * (BN / 32) * KG * 64) void matmul_small_kernel(MatmulArgs g) {
    constexpr int WN = BN / 32, WAVES = BM / 32 * WN * KG, NT = WAVES * 64;
    constexpr int BK = KG * 64, CPR = BK / 16, ROWS = BM + BN, LD = ROWS * CPR / NT;
    static_assert(KG >= 2 && ROWS * CPR % NT == 0 && NT % CPR == 0);
    constexpr int BUFS = DMA ? STAGES : 2, RED = KG * BM * BN / 4;  // 16-byte places
    __shared__ __align__(1024) i32x4 lds[BUFS * ROWS * CPR > RED ? BUFS * ROWS * CPR : RED];
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
    for (int i = 0; i < LD; ++i) src[i] = source(i) + chunk * 16;

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
    auto compute = [&](int buf) {
        const i32x4* A = &lds[buf * ROWS * CPR + wm * 32 * CPR];
        const i32x4* W = &lds[buf * ROWS * CPR + (BM + wn * 32) * CPR];
        i32x4 fa[2], fw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) fw[i] = W[i * 16 * CPR + place], fa[i] = A[i * 16 * CPR + place];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma_i8(fw[j], fa[i], acc[i][j]);
    };
    if constexpr (DMA) {
        auto fetch = [&](int s, int buf) {
#pragma unroll
            for (int i = 0; i < LD; ++i)
                copy_to_lds(src[i] + s * BK, &lds[buf * ROWS * CPR + i * NT + wave * 64]);
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            if (s < full) fetch(s, s);
        int buf = 0;
        for (int s = 0; s < full; ++s) {
            if (s + STAGES - 2 < full)
                wait_vmcnt<(STAGES - 2) * LD>();
            else
                wait_vmcnt<0>();
            lds_barrier();
            if (s + STAGES - 1 < full) fetch(s + STAGES - 1, buf == 0 ? STAGES - 1 : buf - 1);
            compute(buf);
            buf = buf + 1 == STAGES ? 0 : buf + 1;
        }
    } else {
        i32x4 hold[REGS][LD];
        auto load = [&](int s, i32x4(&h)[LD]) {
#pragma unroll
            for (int i = 0; i < LD; ++i) __builtin_memcpy(&h[i], src[i] + s * BK, 16);
        };
        auto put = [&](const i32x4(&h)[LD], int buf) {
#pragma unroll
            for (int i = 0; i < LD; ++i) lds[buf * ROWS * CPR + i * NT + tid] = h[i];
        };
        static_assert(REGS % 2 == 0);
#pragma unroll
        for (int s = 0; s < REGS; ++s)
            if (s < full) load(s, hold[s]);
        if (full > 0) put(hold[0], 0);
        for (int s = 0; s < full; s += REGS)
#pragma unroll
            for (int u = 0; u < REGS; ++u) {
                if (s + u >= full) break;
                lds_barrier();
                if (s + u + REGS < full) load(s + u + REGS, hold[u]);
                compute(u % 2);
                if (s + u + 1 < full) put(hold[(u + 1) % REGS], (u + 1) % 2);
            }
    }
    if (partial) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LD; ++i) lds[i * NT + tid] = rest[i];
        __syncthreads();
        compute(0);
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

template <int BM, int BN, int KG, int STAGES, int REGS, bool DMA>
void small(const MatmulArgs& g) {
    const dim3 grid((unsigned)(((int64_t)g.M + BM - 1) / BM * ((g.N + BN - 1) / BN)));
    constexpr int NT = BM / 32 * (BN / 32) * KG * 64;
    if (g.out_bf16)
        hipLaunchKernelGGL((matmul_small_kernel<BM, BN, KG, STAGES, REGS, DMA, true>), grid, dim3(NT), 0, g.stream, g);
    else
        hipLaunchKernelGGL((matmul_small_kernel<BM, BN, KG, STAGES, REGS, DMA, false>), grid, dim3(NT), 0, g.stream, g);
}

template <int BM, int BN, int WM, int WN, int STAGES, bool DMA>
void tiles(const MatmulArgs& g) {
    const dim3 grid((unsigned)(((int64_t)g.M + BM - 1) / BM * ((g.N + BN - 1) / BN)));
    if (g.out_bf16)
        hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, STAGES, DMA, true>), grid, dim3(WM * WN * 64), 0, g.stream, g);
    else
        hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, STAGES, DMA, false>), grid, dim3(WM * WN * 64), 0, g.stream, g);
}

bool words_ok(const MatmulArgs& g) {
    return ((reinterpret_cast<uintptr_t>(g.a) | reinterpret_cast<uintptr_t>(g.w)) & 3u) == 0 &&
           (g.M == 1 || g.a_stride % 4 == 0) && (g.N == 1 || g.w_stride % 4 == 0);
}

bool dma_ok(const int8_t* p, int64_t stride, int rows, int K) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 &&
           (rows == 1 || (stride % 16 == 0 && stride <= (INT32_MAX - K) / 255));
}

// Form of a product and its expected time: the number of rounds over the 256 CUs (whole ones up to
// 1024 tiles, where they stay in step) times what a tile takes: a fixed part (filling the pipeline, storing)
// and a part for each reduction byte, by how fast a CU brings BM + BN rows in (50 to 70 bytes a
// ns) or, for 256 x 256, multiplies them.  Constants fitted to measurements, M x N x K in us:
//                        32x64  128x64  128x128 (4 / 2 stages)  256x256
//      32 x 12288 x 4096  11.9    14.5     17.3 /  22.5           42.2
//     128 x  4096 x 4096   9.8    13.7     17.1 /  22.9           42.3
//     512 x  4096 x 4096  24.0    16.1     19.2 /  24.1           44.5
//    1024 x  4096 x 4096  48.5    24.6     21.1 /  26.2           46.1
//     512 x 12288 x 4096  62.1    35.6     36.9 /  32.1           50.0
//    2048 x  4096 x 4096  97.2    46.6     41.2 /  35.8           50.5
//    4096 x  4096 x 1024  71.9    32.5     29.8 /  25.2           23.6
//    8192 x  8192 x  512         107.7    114.8 /  85.5           77.1
//    3000 x  4096 x 4096          68.4     57.6 /  59.9           50.3
//    8192 x  2048 x 8192   335     192      158 /   142            118
// (64 x 32 tiles take what 32 x 64 take.)
// The form without tiles is faster where 16 x 16 outputs do not make more than one workgroup for
// each CU (51 x 256 x 8100 8.6 against 17.3 us; at 64 x 2048 x 1024, twice that, 5.3 against 5.1)
// and up to 16 rows and 8192 columns (1 x 4096 x 4096 6.5 against 8.8 us; 1 x 12288 x 4096 12.6
// against 11.1).
enum class Form { rows, t32x64, t128x64, t128x128_deep, t128x128, t256x256 };
struct Plan {
    Form form;
    double us;
};
Plan plan(int64_t M, int64_t N, int K) {
    if ((M <= 16 && N <= 8192) || (M + 15) / 16 * ((N + 15) / 16) <= 256) return Plan{Form::rows, 1.0 + 1.3e-3 * K};
    Plan best{Form::t32x64, 1e30};
    auto offer = [&](Form f, int bm, int bn, int64_t least, int64_t most, double fixed, double per_k) {
        const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
        if (tiles < least || tiles > most) return;
        const double rounds = tiles <= 1024 ? (double)((tiles + 255) / 256) : tiles / 256. + .5;
        const double us = rounds * (fixed + per_k * K * 1e-3);
        if (us < best.us) best = Plan{f, us};
    };
    constexpr int64_t any = (1 << 23) - 1;  // a launch has fewer than 2^32 threads, 512 for each tile
    offer(Form::t32x64, 32, 64, 1, any, 0.8, 1.9);
    offer(Form::t128x64, 128, 64, 1, any, 1.0, 2.8);
    offer(Form::t128x128_deep, 128, 128, 1, 256, 1.8, 4.2);
    offer(Form::t128x128, 128, 128, 257, any, 1.8, 3.6);
    // up to one tile for each CU, a tile takes longer the more of them draw on memory and power
    const double fill = std::min(1.0, ((M + 255) / 256) * ((N + 255) / 256) / 256.0);
    offer(Form::t256x256, 256, 256, 1, any, 8.0, 8.0 + 3.5 * fill * fill);
    return best;
}

template <bool DMA>
void start(Form f, const MatmulArgs& g) {
    switch (f) {
        case Form::rows: words_ok(g) ? g.K % 16 == 0 ? rows<16>(g) : rows<4>(g) : rows<1>(g); break;
        case Form::t32x64: small<32, 64, 4, 3, 4, DMA>(g); break;
        case Form::t128x64: tiles<128, 64, 4, 2, 3, DMA>(g); break;
        case Form::t128x128_deep: tiles<128, 128, 2, 4, DMA ? 4 : 2, DMA>(g); break;
        case Form::t128x128: tiles<128, 128, 2, 4, 2, DMA>(g); break;
        case Form::t256x256: tiles<256, 256, 2, 4, 2, DMA>(g); break;
    }
}

}  // namespace

hipError_t launch_matmul_i8(const MatmulArgs& g) {
    if (g.M < 1 || g.M > GDR_I8_MAX_ROWS || g.N < 1 || g.K < 1 || g.K > GDR_MATMUL_I8_MAX_K) return hipErrorInvalidValue;
    const bool dma = dma_ok(g.a, g.a_stride, g.M, g.K) && dma_ok(g.w, g.w_stride, g.N, g.K);
    const Plan whole = plan(g.M, g.N, g.K);
    // A few rows past a multiple of 256 can cost a round of tiles more: they go into a launch of
    // their own where that is expected to be faster (4097 x 12288 x 4096: 200 against 218 us).
    const int rest = g.M % 256, head = g.M - rest;
    if (head > 0 && rest > 0) {
        const Plan first = plan(head, g.N, g.K), second = plan(rest, g.N, g.K);
        if (first.us + second.us + 3.0 < whole.us) {
            MatmulArgs a = g, b = g;
            a.M = head;
            b.M = rest;
            b.a += head * g.a_stride;
            b.a_scale += head;
            for (int i = 0; i < g.out.n; ++i)
                b.out.ptr[i] = static_cast<char*>(g.out.ptr[i]) + head * g.out.stride[i] * (g.out_bf16 ? 2 : 4);
            dma ? start<true>(first.form, a) : start<false>(first.form, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            dma ? start<true>(second.form, b) : start<false>(second.form, b);
            return hipGetLastError();
        }
    }
    dma ? start<true>(whole.form, g) : start<false>(whole.form, g);
    return hipGetLastError();
}

}  // namespace gdr

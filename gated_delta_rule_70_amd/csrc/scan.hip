// Selective scan: the recurrence with a diagonal transition that depends on the input
// (gdr_selective_scan, gdr_selective_scan_step).
//
//   h[n] <- exp(step A[n]) h[n] + step x B[n],   y = sum_n C[n] h[n]
//
// for every channel.  A differs from channel to channel and state to state, so there is no matrix
// product in it: an exponential, three multiplications and two additions for each token, channel and
// state, in fp32 on the vector ALU.  States never leave fp32, outputs are rounded once, as they are stored.
//
// Prompts are bound by that: for each token and wave of 64 states six cycles of four (the exponential two),
// a token's softplus, gate and sum over its states on top.  us from one call to the next (inputs from
// memory): 4097 tokens of 4096 channels of 16, bf16, 105 (114), where a copy of the inputs and
// outputs would take 27; 8 sequences of 512 70 (76); 4097 x 1024 49 (49); 32768 x 4096 850.  At eight packed sequences
// of 4096 channels the ALU issued in 94 % of the cycles.  fp32 matrix instructions do not run beside the ALU here: one
// of 4 x 4 x 1 takes as long as 3.6 additions, so neither step x B nor the sums over states gain by them.  Single tokens
// are bound by the states' bytes: 256 sequences of 4096 x 16 27 us (31 from memory, 4.6 TB/s).
#include "layer_launch.h"

#include <type_traits>
#include <utility>

#include "row_device.h"

namespace gdr {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(v); }

// Four values as loaded, turned to fp32 where they are used, so that the load stays in flight.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
    f32x4 v;
    __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <>
struct Raw4<bf16_t> {
    u32x2 v;
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    }
};
// Values 0 .. 3 at p, zeros from n on; any alignment.
template <typename T>
__device__ __forceinline__ Raw4<T> load4(const T* p, int n) {
    Raw4<T> r{};
    if (n >= 4) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else if (n > 0) {
        T t[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) t[i] = p[i];
        __builtin_memcpy(&r, t, sizeof(r));
    }
    return r;
}
__device__ __forceinline__ void store4(float* p, int n, f32x4 v) {
    if (n >= 4) {
        __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = v[i];
    }
}
__device__ __forceinline__ void store4(bf16_t* p, int n, f32x4 v) {
    const u32x2 u = bf16x4_bits(v);
    if (n >= 4) {
        __builtin_memcpy(p, &u, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i].bits = (uint16_t)(u[i / 2] >> (i % 2 * 16));
    }
}

// A in units of log2, within the finite values: an infinite one is the same for every step but zero, which
// tokens past a sequence's end have.
__device__ __forceinline__ float rate(float a) {
    constexpr float most = 3.402823466e38f;
    a *= kLog2e;
    return a < -most ? -most : a > most ? most : a;
}

// ---- single tokens -------------------------------------------------------------------------------

// P lanes for each channel (a power of two, at least N / 4), four state values in each, and Q sequences one
// after the other, whose loads are all on their way at once.  Where N is no multiple of four the last
// lane has the last four values, some of them twice: the lanes of a channel are in one wave, so all have read
// before any writes.  (FOURS: N is a multiple; looking at N around the loads costs 256 x 4096 x 16 from memory
// 35 us instead of 31.)  Bound by the states' bytes.
template <typename TX, typename TDT, int P, int Q, bool FOURS>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(ScanArgs a, int tiles, int64_t block0) {
    const int64_t b = block0 + blockIdx.x;
    const int64_t seq0 = b / tiles * Q;
    const int lane = threadIdx.x % P;
    const int d = (int)(b % tiles) * (kThreads / P) + threadIdx.x / P;
    if (d >= a.D) return;  // all lanes of a channel
    const int N = a.N, most = FOURS ? 4 : N;
    const int n = FOURS ? 4 * lane : N < 4 ? 0 : min(4 * lane, N - 4), twice = 4 * lane - n, g = a.G == 1 ? 0 : d / (a.D / a.G);
    const bool mine = 4 * lane < N;
    Raw4<float> h[Q], A{};
    Raw4<TX> B[Q], C[Q];
    TX x[Q], z[Q];
    TDT dt[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int64_t seq = seq0 + q < a.B ? seq0 + q : a.B - 1;  // past the last one: loaded again, not stored
        h[q] = Raw4<float>{};
        B[q] = C[q] = Raw4<TX>{};
        if (mine) {
            if (a.h0) h[q] = load4(a.h0 + (seq * a.D + d) * N + n, most);
            B[q] = load4(static_cast<const TX*>(a.b) + seq * a.b_stride + (int64_t)g * N + n, most);
            C[q] = load4(static_cast<const TX*>(a.c) + seq * a.c_stride + (int64_t)g * N + n, most);
        }
        x[q] = static_cast<const TX*>(a.x)[seq * a.x_stride + d];
        dt[q] = static_cast<const TDT*>(a.dt)[seq * a.dt_stride + d];
        z[q] = a.z ? static_cast<const TX*>(a.z)[seq * a.z_stride + d] : TX{};
    }
    if (mine) A = load4(a.A + (int64_t)d * N + n, most);
    const float skip = a.skip ? a.skip[d] : 0.f, bias = a.dt_bias ? a.dt_bias[d] : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (seq0 + q >= a.B) return;
        float step = to_f32(dt[q]) + bias;
        if (a.softplus) step = softplus(step);
        const float xv = to_f32(x[q]), in = step * xv;
        f32x4 v;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(step * rate(A.get(i))), h[q].get(i), in * B[q].get(i));
            y = !FOURS && (i < twice || n + i >= N) ? y : __builtin_fmaf(C[q].get(i), v[i], y);
        }
        if (mine && a.ht) store4(a.ht + ((seq0 + q) * a.D + d) * N + n, most, v);
        if (!mine) y = 0.f;  // an infinite step x times its B and C of zero is none
        if constexpr (P > 1) y += dpp_mov<0xB1>(y);   // quad_perm [1,0,3,2]
        if constexpr (P > 2) y += dpp_mov<0x4E>(y);   // quad_perm [2,3,0,1]
        if constexpr (P > 4) y += dpp_mov<0x141>(y);  // row_half_mirror
        if constexpr (P > 8) y += dpp_mov<0x140>(y);  // row_mirror
        if constexpr (P > 16) y += __shfl_xor(y, 16);
        if (a.skip) y = __builtin_fmaf(skip, xv, y);  // not 0 x, which is NaN where x is infinite
        TX* out = static_cast<TX*>(a.out) + (seq0 + q) * a.out_stride + d;
        if (a.z) y *= silu_for(to_f32(z[q]), out);
        if (lane == 0) store1(out, y);
    }
}

// ---- prompts -------------------------------------------------------------------------------------

// Lane J's value in all L lanes that share a channel.
template <int L, int J>
__device__ __forceinline__ float broadcast(float x) {
    static_assert(L == 16 || L == 4, "a row of lanes, or a quad");
    return dpp_mov<L == 16 ? 0x150 + J : J * 0x55>(x);  // row_newbcast, quad_perm
}

// The sums over L lanes of L values each, lane j having the j-th: lanes exchange halves of what they
// hold, opposite ones first.
template <int L>
__device__ __forceinline__ float sum_scatter(float (&p)[L], int lane) {
    if constexpr (L == 16) {
        // The halves are lanes of four banks each, so an addition to some banks only makes the choice: two
        // instructions for a value instead of three.  s_nop: a DPP operand must be two cycles old.
        float r[8], q[4];
        asm("s_nop 1\n"
            "v_add_f32_dpp %0, %8, %8 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %0, %16, %16 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %1, %9, %9 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %1, %17, %17 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %2, %10, %10 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %2, %18, %18 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %3, %11, %11 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %3, %19, %19 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %4, %12, %12 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %4, %20, %20 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %5, %13, %13 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %5, %21, %21 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %6, %14, %14 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %6, %22, %22 row_mirror row_mask:0xf bank_mask:0xc\n"
            "v_add_f32_dpp %7, %15, %15 row_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %7, %23, %23 row_mirror row_mask:0xf bank_mask:0xc\n"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
            : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(p[4]), "v"(p[5]), "v"(p[6]), "v"(p[7]), "v"(p[8]), "v"(p[9]), "v"(p[10]), "v"(p[11]), "v"(p[12]), "v"(p[13]), "v"(p[14]), "v"(p[15]));
        asm("s_nop 1\n"
            "v_add_f32_dpp %0, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %0, %8, %8 row_half_mirror row_mask:0xf bank_mask:0xa\n"
            "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %1, %9, %9 row_half_mirror row_mask:0xf bank_mask:0xa\n"
            "v_add_f32_dpp %2, %6, %6 row_half_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %2, %10, %10 row_half_mirror row_mask:0xf bank_mask:0xa\n"
            "v_add_f32_dpp %3, %7, %7 row_half_mirror row_mask:0xf bank_mask:0xf\n"
            "v_add_f32_dpp %3, %11, %11 row_half_mirror row_mask:0xf bank_mask:0xa\n"
            : "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3])
            : "v"(r[0]), "v"(r[1]), "v"(r[2]), "v"(r[3]), "v"(r[4]), "v"(r[5]), "v"(r[6]), "v"(r[7]));
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = q[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = lane & 2 ? p[i + 2] : p[i], send = lane & 2 ? p[i] : p[i + 2];
        p[i] = keep + dpp_mov<0x1B>(send);  // quad_perm [3,2,1,0]
    }
    const float keep = lane & 1 ? p[1] : p[0], send = lane & 1 ? p[0] : p[1];
    return keep + dpp_mov<0xB1>(send);  // quad_perm [1,0,3,2]
}

template <int... J, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, J...>, F f) {
    (f(std::integral_constant<int, J>{}), ...);
}

// A workgroup runs CT channels of one sequence from its first token to its last, TT tokens a tile.
// L lanes share a channel, S state values in each, in registers throughout.  A tile's step and x lie
// in LDS as [token][channel], B and C as [state][token] (L = 16) or [token][state] (L = 4), the next
// tile's are on their way in registers meanwhile.  In a chunk of L tokens lane j reads the j-th
// token's step and x and hands them to the others (DPP), and each lane sums its own states' part of
// y for every token; sum_scatter leaves the j-th token's y in lane j.
//
// Half of the waves do nothing but that; the others load, compute steps, and gate and store a tile behind.
// With one set of waves for all of it, 4097 x 4096 x 16 took 160 us instead of 113 (105 since) and 8 x 4096 x 4096 725
// instead of 556: a wave that is alone on its SIMD issues every 5 to 6 cycles at best.  Leaving the sums over lanes to
// the storing waves too (parts of y through LDS) took 127.  Tiles of 32 tokens instead of 64 took 195 (memory's
// latency shows), TT = 48 for S = 4 263 instead of 291 (N = 64).
template <int L, int S>
struct Tile {
    static constexpr int CT = kThreads / L;
    static constexpr int TT = scan_tile_tokens(L, S);
    static constexpr int NP = L * S;                                         // places for states
    static constexpr int bc = L == 16 ? NP * (TT + 4) : TT * NP;
    static constexpr int groups = (TT * CT / 4 + kThreads - 1) / kThreads;   // of four channels, for a thread to bring
    static constexpr int bc_groups = (TT * NP / 4 + kThreads - 1) / kThreads;  // of four states
    // Where token t's state n lies (L = 16: the states of neighbouring lanes in neighbouring rows, which
    // are four words apart in their banks).
    static __device__ __forceinline__ int at_state(int t, int n) {
        return L == 16 ? (n % S * 16 + n / S) * (TT + 4) + t : t * NP + n;
    }
    // Where token t's channel c lies: channels are exchanged in fours so that the lanes of a wave,
    // on L tokens of 64 / L channels, read 64 words that differ modulo 64.  (The counters have 0.5 to 0.9 cycles of
    // bank conflicts for each LDS instruction all the same, 1.7 in the launch for the states behind segments.)
    static __device__ __forceinline__ int at(int t, int c) {
        return t * CT + (c ^ (L == 16 ? (t >> 2 & 3) << 2 : (t & 3) << 4));
    }
};

// Which of a channel's N states is in each of its NP places, where they are more.  A place without a state would
// hold zeros, and an infinite input times those is NaN, in the sum y too; so every place has one.  States go in
// fours (as they are brought), the last four possibly beginning earlier: each four 2^k times, and the first
// `more` of them as often again, which makes every state's copies a power of two.  Its C is divided by their
// number, and their parts of y add up to its own exactly.  (The last fours that share states are there equally
// often: fours + more is even, so `more` never ends between them.)  4097 x 4096 us with copies / zeros in those
// places: N = 10 106 / 106, 20 148 / 149, 48 264 / 263, 100 555 / 528.
struct Places {
    int N, fours, k, more;
    __device__ __forceinline__ Places(int n, int np) : N(n), fours((n + 3) / 4), k(0) {
        while (2 * fours << k <= np / 4) ++k;
        more = (np / 4 >> k) - fours;
    }
    // The first state of the four in places 4 g to 4 g + 3.
    __device__ __forceinline__ int first(int g) const {
        const int w = g >> k;
        return N < 4 ? 0 : min(4 * (w < fours ? w : w - fours), N - 4);
    }
    __device__ __forceinline__ int state(int place) const {
        const int j = place % 4;
        return N < 4 ? j < N ? j : N == 2 ? j - 2 : 0 : first(place / 4) + j;
    }
    // Fewer than four states in four places, as `state` has them; what belongs to a copy is that of the state.
    __device__ __forceinline__ f32x4 repeat(f32x4 v) const {
        return f32x4{v[0], N == 1 ? v[0] : v[1], N < 3 ? v[0] : v[2], N == 2 ? v[1] : v[0]};
    }
    // Whether it is the first copy of its four.
    __device__ __forceinline__ bool own(int place) const {
        const int g = place / 4;
        return g < fours << k && g % (1 << k) == 0;
    }
    __device__ __forceinline__ float share(int state) const {
        const int w = state / 4, last = 1 << k << (fours - 1 < more);
        const int copies = N < 4 ? (N == 3 ? 1 + (state == 0) : 4 / N) << k
                                 : (w < fours - 1 ? 1 << k << (w < more) : 0) + (state >= N - 4 ? last : 0);
        return __builtin_ldexpf(1.f, -__builtin_ctz(copies));
    }
};

// What a launch does: whole sequences, or sequences cut into segments of a.seg_len tokens, the
// states behind each first (from zero, without outputs), then each segment from its start.  The first
// launch also puts h0 by: ht may be h0, and the second one's last segment writes it while others begin.
enum { kWhole, kEnds, kSegments };

// First slot of a packed batch's sequence i: strictly ascending, fewer than T / seg_len + B.
__device__ __forceinline__ int64_t packed_slot(const ScanArgs& a, int i) {
    return min(max(a.cu[i], 0), a.T) / a.seg_len + i;
}

// COPIES: N states are fewer than places.
template <typename TX, typename TDT, int L, int S, int MODE, bool COPIES>
__global__ __launch_bounds__(2 * kThreads, S <= 4 ? 4 : 2) void scan_kernel(ScanArgs a, int tiles, int64_t block0) {
    using K = Tile<L, S>;
    constexpr int CT = K::CT, TT = K::TT, NP = K::NP;
    __shared__ __align__(16) float sDt[2][TT * CT], sX[2][TT * CT], sY[2][TT * CT];
    __shared__ __align__(16) float sB[2][K::bc], sC[2][K::bc];
    static_assert(K::bc % 4 == 0);

    const int64_t b = block0 + blockIdx.x;
    const int64_t slot = b / (tiles * a.G);  // sequence, and segment
    // each sequence on all XCDs, neighbouring channels, whose values share lines, on one
    const int gt = (int)xcd_order(b % (tiles * a.G), tiles * a.G);
    int seq = (int)slot, seg = 0;
    if (MODE != kWhole) {
        seq = (int)(slot / a.segs), seg = (int)(slot % a.segs);
        if (a.cu) {  // the last sequence whose slots begin at or before this one
            int hi = a.B - 1;
            seq = 0;
            while (seq < hi) {
                const int mid = (seq + hi + 1) >> 1;
                if (packed_slot(a, mid) <= slot)
                    seq = mid;
                else
                    hi = mid - 1;
            }
            seg = (int)(slot - packed_slot(a, seq));
            if (seg < 0) return;  // before the first row
        }
    }
    const int g = gt / tiles, per = a.D / a.G, c0 = gt % tiles * CT;  // first channel in the group
    const int d0 = g * per + c0, left = per - c0;                     // in all; channels from there on
    int64_t first = (int64_t)seq * a.T;
    int len = a.T;
    if (a.cu) {
        const Span s = packed_span(a.cu, seq, a.T);
        first = s.first, len = s.count;
    }
    bool last = true;  // segment of the sequence
    int64_t begin = seq;  // where its first state lies
    if constexpr (MODE != kWhole) {
        const int64_t behind = (int64_t)seg * a.seg_len;
        if (seg > 0 && behind >= len) return;
        last = behind + a.seg_len >= len;
        if (MODE == kEnds && last) {  // no segment starts from it; its place holds h0 for the others
            const int64_t from = (int64_t)seq * a.D + d0, to = slot * a.D + d0, n = (int64_t)min(CT, left) * a.N;
            for (int64_t i = threadIdx.x; a.h0 && i < n; i += 2 * kThreads) a.workspace[to * a.N + i] = a.h0[from * a.N + i];
            return;
        }
        if (MODE == kSegments) begin = slot - seg + (len > 0 ? (len - 1) / a.seg_len : 0);
        first += behind;
        len = last ? len - (int)behind : a.seg_len;
    }
    const int tid = threadIdx.x % kThreads, N = a.N;
    const Places places(N, NP);
    if constexpr (MODE == kEnds) {  // has no sums: places past N only need to hold something
        for (int i = threadIdx.x; i < K::bc; i += 2 * kThreads) sB[0][i] = sB[1][i] = 0.f;
        lds_barrier();
    }

    if (threadIdx.x >= kThreads) {
        // What this thread brings of a tile: groups of four channels, of tokens rowsApart from each other,
        // and of four states of B and C.
        constexpr int rowsApart = kThreads / (CT / 4), bcApart = kThreads / (NP / 4);
        const int gc = tid % (CT / 4) * 4, gt0 = tid / (CT / 4), gn = left - gc;
        const TX* x = static_cast<const TX*>(a.x) + (first + gt0) * a.x_stride + d0 + gc;
        const TDT* dt = static_cast<const TDT*>(a.dt) + (first + gt0) * a.dt_stride + d0 + gc;
        const TX* z = a.z && MODE != kEnds ? static_cast<const TX*>(a.z) + (first + gt0) * a.z_stride + d0 + gc : nullptr;
        TX* out = static_cast<TX*>(a.out) + (first + gt0) * a.out_stride + d0 + gc;
        // the last four states where N is no multiple of four: some are then brought twice
        const int bt = tid / (NP / 4), group = tid % (NP / 4) * 4, bn = COPIES ? places.first(group / 4) : N < 4 ? group : min(group, N - 4);
        const bool brings = COPIES || group < N;
        float share[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) share[j] = COPIES ? places.share(places.state(group + j)) : 1.f;
        const TX* B = static_cast<const TX*>(a.b) + (first + bt) * a.b_stride + (int64_t)g * N + bn;
        const TX* C = static_cast<const TX*>(a.c) + (first + bt) * a.c_stride + (int64_t)g * N + bn;
        struct Held {  // of a tile, on its way
            Raw4<TX> x[K::groups], b[K::bc_groups], c[K::bc_groups];
            Raw4<TDT> dt[K::groups];
        } held[2];
        Raw4<TX> gates[2][K::groups];
        float bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[i] = a.dt_bias && i < gn ? a.dt_bias[d0 + gc + i] : 0.f;

        // Tiles of nothing but whole groups are loaded and stored without looking at their ends: a branch
        // around a load makes the next instructions wait for it.
        const bool whole = left >= CT && N >= 4;
        auto bring = [&](int t0, Held& r) {  // the tile at t0, on which the pointers stand
            if (t0 >= len) return;
            if (whole && t0 + TT <= len) {
#pragma unroll
                for (int i = 0; i < K::groups; ++i)
                    if (rowsApart * K::groups == TT || gt0 < TT) {
                        r.x[i] = load4(x + i * rowsApart * a.x_stride, 4);
                        r.dt[i] = load4(dt + i * rowsApart * a.dt_stride, 4);
                    }
#pragma unroll
                for (int i = 0; i < K::bc_groups; ++i) {
                    r.b[i] = r.c[i] = Raw4<TX>{};
                    if ((bcApart * K::bc_groups == TT || bt < TT) && brings) {
                        r.b[i] = load4(B + i * bcApart * a.b_stride, 4);
                        if constexpr (MODE != kEnds) r.c[i] = load4(C + i * bcApart * a.c_stride, 4);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < K::groups; ++i) {
                    const int t = gt0 + i * rowsApart, n = t < TT && t0 + t < len ? gn : 0;
                    r.x[i] = load4(x + i * rowsApart * a.x_stride, n);
                    r.dt[i] = load4(dt + i * rowsApart * a.dt_stride, n);
                }
#pragma unroll
                for (int i = 0; i < K::bc_groups; ++i) {
                    const int t = bt + i * bcApart, n = brings && t < TT && t0 + t < len ? N - bn : 0;
                    r.b[i] = load4(B + i * bcApart * a.b_stride, n);
                    if constexpr (MODE != kEnds) r.c[i] = load4(C + i * bcApart * a.c_stride, n);
                }
            }
            x += TT * a.x_stride;
            dt += TT * a.dt_stride;
            B += TT * a.b_stride;
            C += TT * a.c_stride;
        };
        auto stage = [&](int t0, int buf, const Held& r) {
            if (t0 >= len) return;
#pragma unroll
            for (int i = 0; i < K::groups; ++i) {
                const int t = gt0 + i * rowsApart;
                if (t >= TT) break;
                f32x4 sv, xv;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sv[j] = r.dt[i].get(j) + bias[j];
                    xv[j] = r.x[i].get(j);
                }
                if (a.softplus)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sv[j] = softplus(sv[j]);
                if (t0 + t >= len) sv = f32x4{0.f, 0.f, 0.f, 0.f};  // tokens past the end leave the state as it is
                *reinterpret_cast<f32x4*>(&sDt[buf][K::at(t, gc)]) = sv;
                *reinterpret_cast<f32x4*>(&sX[buf][K::at(t, gc)]) = xv;
            }
#pragma unroll
            for (int i = 0; i < K::bc_groups; ++i) {
                const int t = bt + i * bcApart;
                if (t >= TT || !brings) break;
                f32x4 b, c = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[j] = r.b[i].get(j);
                    if constexpr (MODE != kEnds) c[j] = COPIES ? r.c[i].get(j) * share[j] : r.c[i].get(j);
                }
                if (COPIES && NP <= 16 && N < 4) b = places.repeat(b), c = places.repeat(c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int to = COPIES ? K::at_state(t, group + j) : K::at_state(t, bn + j);
                    sB[buf][to] = b[j];
                    if constexpr (MODE != kEnds) sC[buf][to] = c[j];
                }
            }
        };
        auto bring_gate = [&](int t0, Raw4<TX>(&rz)[K::groups]) {
            if (!z || t0 >= len) return;
#pragma unroll
            for (int i = 0; i < K::groups; ++i) {
                const int t = gt0 + i * rowsApart;
                if (whole && t0 + TT <= len) {
                    if (rowsApart * K::groups == TT || gt0 < TT) rz[i] = load4(z + i * rowsApart * a.z_stride, 4);
                } else {
                    rz[i] = load4(z + i * rowsApart * a.z_stride, t < TT && t0 + t < len ? gn : 0);
                }
            }
            z += TT * a.z_stride;
        };
        auto store = [&](int t0, int buf, const Raw4<TX>(&rz)[K::groups]) {
#pragma unroll
            for (int i = 0; i < K::groups; ++i) {
                const int t = gt0 + i * rowsApart;
                if (t >= TT) break;
                f32x4 y = *reinterpret_cast<const f32x4*>(&sY[buf][K::at(t, gc)]);
                if (z)
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] *= silu_for(rz[i].get(j), out);
                if (whole && t0 + TT <= len)
                    store4(out + i * rowsApart * a.out_stride, 4, y);
                else if (t0 + t < len)
                    store4(out + i * rowsApart * a.out_stride, gn, y);
            }
            out += TT * a.out_stride;
        };

        // Two tiles are on their way while one is computed: at 25 ns a token a tile of 64 takes 1.6 us, not
        // much more than memory's latency.
        bring(0, held[0]);
        stage(0, 0, held[0]);
        bring(TT, held[1]);
        bring(2 * TT, held[0]);
        bring_gate(0, gates[0]);
        lds_barrier();
        auto pass = [&](int t0, auto parity) {
            constexpr int P = decltype(parity)::value;
            if (MODE != kEnds && t0 > 0) store(t0 - TT, P ^ 1, gates[P ^ 1]);
            bring_gate(t0 + TT, gates[P ^ 1]);
            stage(t0 + TT, P ^ 1, held[P ^ 1]);
            bring(t0 + 3 * TT, held[P ^ 1]);
            lds_barrier();
        };
#pragma unroll 1
        for (int t0 = 0; t0 < len; t0 += 2 * TT) {
            pass(t0, std::integral_constant<int, 0>{});
            if (t0 + TT < len) pass(t0 + TT, std::integral_constant<int, 1>{});
        }
        if (MODE != kEnds && len > 0) {
            const int end = (len - 1) / TT;
            if (end & 1)
                store(end * TT, 1, gates[1]);
            else
                store(end * TT, 0, gates[0]);
        }
        return;
    }

    const int lane = tid % L, c = tid / L;
    const bool mine = c < left;
    float A[S], h[S];
    const int64_t channel = ((int64_t)seq * a.D + d0 + c) * N;
    const float* h0 = a.h0 && MODE != kEnds ? (MODE == kSegments ? a.workspace : a.h0) + (begin * a.D + d0 + c) * N : nullptr;
    int state[S];  // in this lane's places
#pragma unroll
    for (int s = 0; s < S; ++s) state[s] = COPIES ? places.state(lane * S + s) : lane * S + s;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const bool there = mine && state[s] < N;
        A[s] = there && len > 0 ? rate(a.A[(int64_t)(d0 + c) * N + state[s]]) : 0.f;
        h[s] = there && h0 ? h0[state[s]] : 0.f;
    }
    const float skip = mine && a.skip && MODE != kEnds ? a.skip[d0 + c] : 0.f;
    // The state behind a segment, from zero, and its sum of steps lie in the workspace, [slot][D][N] and
    // [slot][D]: with them the state before this segment follows from the sequence's first one.  A hundred
    // segments are a chain of loads unless several are asked for together (B 1, T 6468, D 64, N 16: 38 us
    // one by one, 22 us eight at a time).
    float* const ends = a.workspace;
    float* const steps = ends + (int64_t)a.B * a.segs * a.D * N;
    if constexpr (MODE == kSegments) {
        constexpr int kAtOnce = S <= 2 ? 8 : 2;  // few states a lane: the registers are there
        for (int64_t e0 = slot - seg; mine && e0 < slot; e0 += kAtOnce) {
            float sums[kAtOnce], end[kAtOnce][S];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int64_t e = e0 + i < slot ? e0 + i : e0;
                sums[i] = steps[e * a.D + d0 + c];
#pragma unroll
                for (int s = 0; s < S; ++s) end[i][s] = state[s] < N ? ends[(e * a.D + d0 + c) * N + state[s]] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (e0 + i < slot)
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        // A whole segment's factor may pass fp32's range where the state does not: it is taken in
                        // two halves, finite ones for the sake of a state of zero (a NaN of the steps is in `end`, too).
                        const float half = fminf(__builtin_amdgcn_exp2f(0.5f * sums[i] * A[s]), 3.402823466e38f);
                        h[s] = __builtin_fmaf(half * h[s], half, end[i][s]);
                    }
        }
        // An infinite state stays so, token by token, unless a token's own factor is zero: a segment's whole factor
        // does not tell.  A thread that has come to infinity, or to NaN by zero times it, goes through the segments
        // again and looks.
        bool lost = false;
#pragma unroll
        for (int s = 0; s < S; ++s) lost |= !(fabsf(h[s]) <= 3.402823466e38f);
        if (lost) {
            const TDT* dt = static_cast<const TDT*>(a.dt) + (first - (int64_t)seg * a.seg_len) * a.dt_stride + d0 + c;
            const float bias = a.dt_bias ? a.dt_bias[d0 + c] : 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float v = h0 ? h0[state[s]] : 0.f;
#pragma unroll 1
                for (int i = 0; i < seg; ++i) {
                    const int64_t e = slot - seg + i;
                    const float half = fminf(__builtin_amdgcn_exp2f(0.5f * steps[e * a.D + d0 + c] * A[s]), 3.402823466e38f);
                    const float end = ends[(e * a.D + d0 + c) * N + state[s]];
                    bool stays = fabsf(v) > 3.402823466e38f;
                    float next = stays ? v + end : __builtin_fmaf(half * v, half, end);
#pragma unroll 1
                    for (int t = 0; stays && t < a.seg_len; ++t) {
                        float step = to_f32(dt[((int64_t)i * a.seg_len + t) * a.dt_stride]) + bias;
                        if (a.softplus) step = softplus(step);
                        if (__builtin_amdgcn_exp2f(step * A[s]) == 0.f) stays = false, next = __builtin_nanf("");
                    }
                    v = next;
                }
                h[s] = v;
            }
        }
    }
    // What was loaded so far is waited for here: left to its first use in the loop, the wait would be
    // there in every pass.
#pragma unroll
    for (int s = 0; s < S; ++s) asm volatile("" : "+v"(A[s]), "+v"(h[s]));

    // B and C of four tokens for this lane's states
    struct Four {
        f32x4 b[S], c[S];
    };
    auto four = [&](int buf, int t, Four& f) {
        if constexpr (L == 16) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                f.b[s] = *reinterpret_cast<const f32x4*>(&sB[buf][(s * 16 + lane) * (TT + 4) + t]);
                if constexpr (MODE != kEnds) f.c[s] = *reinterpret_cast<const f32x4*>(&sC[buf][(s * 16 + lane) * (TT + 4) + t]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float b[S], cc[S];
                __builtin_memcpy(b, __builtin_assume_aligned(&sB[buf][(t + i) * NP + lane * S], 4 * S), sizeof(b));
                if constexpr (MODE != kEnds) __builtin_memcpy(cc, __builtin_assume_aligned(&sC[buf][(t + i) * NP + lane * S], 4 * S), sizeof(cc));
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    f.b[s][i] = b[s];
                    if constexpr (MODE != kEnds) f.c[s][i] = cc[s];
                }
            }
        }
    };
    float sum = 0.f;  // of this lane's steps
    auto compute = [&](int buf) {
        // operands from LDS are read one group of four tokens (step and x one chunk) ahead, into two
        // sets of registers in turn
        constexpr int chunks = L == 16 ? 1 : 2;  // of a pass, so that it has an even number of groups
        Four f[2];
        four(buf, 0, f[0]);
        float step = sDt[buf][K::at(lane, c)], xv = sX[buf][K::at(lane, c)];
#pragma unroll 1
        for (int t0 = 0; t0 < TT; t0 += chunks * L) {
#pragma unroll
            for (int k = 0; k < chunks; ++k) {
                const int here = t0 + k * L;
                const int after = here + L < TT ? here + L : 0;  // nothing is done with what is read behind the last chunk
                const float step1 = sDt[buf][K::at(after + lane, c)], xv1 = sX[buf][K::at(after + lane, c)];
                const float in = step * xv;
                if constexpr (MODE == kEnds) sum += step;
                float p[L];
                unrolled(std::make_integer_sequence<int, L>{}, [&](auto j) {
                    constexpr int J = decltype(j)::value;
                    Four &now = f[(k * (L / 4) + J / 4) % 2], &next = f[(k * (L / 4) + J / 4 + 1) % 2];
                    if constexpr (J % 4 == 0) four(buf, J + 4 < L ? here + J + 4 : after, next);
                    const float sj = broadcast<L, J>(step), ij = broadcast<L, J>(in);
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        h[s] = __builtin_fmaf(__builtin_amdgcn_exp2f(sj * A[s]), h[s], ij * now.b[s][J % 4]);
                        if constexpr (MODE != kEnds) p[J] = s ? __builtin_fmaf(now.c[s][J % 4], h[s], p[J]) : now.c[s][J % 4] * h[s];
                    }
                });
                if constexpr (MODE != kEnds) {
                    const float y = sum_scatter<L>(p, lane);
                    sY[buf][K::at(here + lane, c)] = a.skip ? __builtin_fmaf(skip, xv, y) : y;
                }
                step = step1, xv = xv1;
            }
        }
    };

    lds_barrier();
#pragma unroll 1
    for (int t0 = 0, buf = 0; t0 < len; t0 += TT, buf ^= 1) {
        compute(buf);
        lds_barrier();
    }
    if constexpr (MODE == kEnds) {
        sum += dpp_mov<0xB1>(sum);  // quad_perm [1,0,3,2]
        sum += dpp_mov<0x4E>(sum);  // quad_perm [2,3,0,1]
        if constexpr (L == 16) {
            sum += dpp_mov<0x141>(sum);  // row_half_mirror
            sum += dpp_mov<0x140>(sum);  // row_mirror
        }
        if (mine) {
            if (lane == 0) steps[slot * a.D + d0 + c] = sum;
            float* end = ends + (slot * a.D + d0 + c) * N + lane * S;
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (lane * S + s < N) end[s] = h[s];
        }
    } else if (a.ht && mine && last) {
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (COPIES ? places.own(lane * S + s) : lane * S + s < N) a.ht[channel + state[s]] = h[s];
    }
}

bool valid(const ScanArgs& a) {
    return a.B >= 1 && a.D >= 1 && a.N >= 1 && a.N <= GDR_SCAN_MAX_STATES && a.G >= 1 && a.D % a.G == 0;
}

template <typename TX, typename TDT, int P>
hipError_t launch_step(const ScanArgs& a) {
    constexpr int channels = kThreads / P;
    const int tiles = (a.D + channels - 1) / channels;
    auto go = [&](auto kernel, int q) {
        return by_blocks(((int64_t)a.B + q - 1) / q * tiles, kThreads, [&](int64_t first, unsigned count) {
            hipLaunchKernelGGL(kernel, dim3(count), dim3(kThreads), 0, a.stream, a, tiles, first);
        });
    };
    if (a.N % 4) return go(scan_step_kernel<TX, TDT, P, 1, false>, 1);
    // Two sequences for a workgroup where that leaves enough of them.  us at 1 / 2 / 4, states from memory:
    // 256 x 4096 x 16 34.0 / 31.1 / 30.9, 256 x 4096 x 8 20.1 / 18.4 / 21.5, 128 x 4096 x 16 19.5 / 17.8 / 18.8.
    return (int64_t)a.B * tiles >= 8192 ? go(scan_step_kernel<TX, TDT, P, 2, true>, 2) : go(scan_step_kernel<TX, TDT, P, 1, true>, 1);
}

template <typename TX, typename TDT>
hipError_t launch_step(const ScanArgs& a) {
    if (a.N <= 4) return launch_step<TX, TDT, 1>(a);
    if (a.N <= 8) return launch_step<TX, TDT, 2>(a);
    if (a.N <= 16) return launch_step<TX, TDT, 4>(a);
    if (a.N <= 32) return launch_step<TX, TDT, 8>(a);
    if (a.N <= 64) return launch_step<TX, TDT, 16>(a);
    return launch_step<TX, TDT, 32>(a);
}

template <typename TX, typename TDT, int L, int S>
hipError_t launch_tiles(const ScanArgs& a) {
    constexpr int CT = Tile<L, S>::CT;
    const int tiles = (a.D / a.G + CT - 1) / CT;
    auto go = [&](int64_t slots, auto kernel) {
        return by_blocks(slots * a.G * tiles, 2 * kThreads, [&](int64_t first, unsigned count) {
            hipLaunchKernelGGL(kernel, dim3(count), dim3(2 * kThreads), 0, a.stream, a, tiles, first);
        });
    };
    const bool copies = a.N < L * S;
    if constexpr (L == 16) {
        if (a.segs > 1) {
            const hipError_t e = go((int64_t)a.B * a.segs, scan_kernel<TX, TDT, L, S, kEnds, false>);
            if (e != hipSuccess) return e;
            return go((int64_t)a.B * a.segs, copies ? scan_kernel<TX, TDT, L, S, kSegments, true> : scan_kernel<TX, TDT, L, S, kSegments, false>);
        }
    }
    return go(a.B, copies ? scan_kernel<TX, TDT, L, S, kWhole, true> : scan_kernel<TX, TDT, L, S, kWhole, false>);
}

template <typename TX, typename TDT>
hipError_t launch(const ScanArgs& a) {
    const ScanTile t = scan_tile(a.B, a.D, a.N, a.G, a.cu != nullptr, a.segs);
    if (t.lanes == 4) return t.states == 2 ? launch_tiles<TX, TDT, 4, 2>(a) : launch_tiles<TX, TDT, 4, 4>(a);
    return t.states == 1   ? launch_tiles<TX, TDT, 16, 1>(a)
           : t.states == 2 ? launch_tiles<TX, TDT, 16, 2>(a)
           : t.states == 4 ? launch_tiles<TX, TDT, 16, 4>(a)
                           : launch_tiles<TX, TDT, 16, 8>(a);
}

}  // namespace

hipError_t launch_selective_scan(const ScanArgs& a) {
    if (!valid(a) || a.segs < 1 || (a.segs > 1 && (!a.workspace || a.seg_len < 1))) return hipErrorInvalidValue;
    if (!a.bf16) return launch<float, float>(a);
    return a.dt_bf16 ? launch<bf16_t, bf16_t>(a) : launch<bf16_t, float>(a);
}

hipError_t launch_selective_scan_step(const ScanArgs& a) {
    if (!valid(a)) return hipErrorInvalidValue;
    if (!a.bf16) return launch_step<float, float>(a);
    return a.dt_bf16 ? launch_step<bf16_t, bf16_t>(a) : launch_step<bf16_t, float>(a);
}

}  // namespace gdr

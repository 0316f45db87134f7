// prompt_internal.h -- attention over whole prompts: the arguments of its
// kernels, and the device pieces that the forward and the backward pass share.
// Internal to the library: the public interface is include/gdr_attention.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device_util.h"
#include "gdr_internal.h"
#include "wave.h"

// on lambdas: the compiler leaves large ones, and those on rare paths, as calls,
// with all that they capture in memory
#define GDR_INLINE __attribute__((always_inline))

namespace gdr {

struct PromptArgs {
    const void *q, *k, *v;       // [T_total, Hq, D], [T_total, Hkv, D]
    const int32_t *cu;           // [B+1] or nullptr (T each)
    void *o;                     // [T_total, Hq, D] (backward: read)
    float *lse;                  // [T_total, Hq] or nullptr (backward: read)
    const void *d_o;             // backward only, from here on
    void *dq, *dk, *dv;
    void *ws;
    int B, T, T_total, Hq, Hkv, G;
    float scale;
    int window;                  // 0: none
};
hipError_t launch_attention_prefill(bool bf16_io, int D, const PromptArgs &a, hipStream_t s);
hipError_t launch_attention_backward(bool bf16_io, int D, const PromptArgs &a, hipStream_t s);
size_t attention_backward_workspace(bool bf16_io, int B, int T_total, int Hq, int Hkv, int D);

// the same calls, or parts of them, in blocks of 32 rows (prompt_short.hip)
hipError_t launch_prompt_short(bool bf16_io, int D, const PromptArgs &a, hipStream_t s);
hipError_t launch_queries_short(bool bf16_io, int D, const PromptArgs &a, hipStream_t s);
hipError_t launch_keys_short(bool bf16_io, int D, const PromptArgs &a, hipStream_t s);

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// A block of RB tokens of one sequence: its number in the sequence (-1: there
// is none), the sequence's first row and its tokens.
struct Block { int i, row0, len; };

// Blocks of a batch, numbered over the sequences.  Packed, the blocks of
// sequence b start at cu[b] / RB + b, which leaves each at least as many as it
// has, so that no sums over the sequences before are needed: a few searches of
// 64 lanes over cu find the sequence.
template <int RB>
inline long long block_bound(const PromptArgs &a) {
    return a.cu ? (long long)a.T_total / RB + a.B : (long long)a.B * ((a.T + RB - 1) / RB);
}
// A batch goes sequence by sequence, each one's longest blocks first (of rows the
// last, of tokens (KEYS) the first), which keeps what a sequence's blocks read in
// the XCDs' caches, but for the last `mixed` sequences, of a packed batch all or
// none: of those the longest blocks of all go first, so that no long one is left for
// the end.  Packed, these are found by sums over the sequences, one a lane: of the
// blocks that are longer than t, for a t that halves the range each time.
//   Rows go from the last sequence to the first and tokens, after them, from the
// first on, of which most is still in the caches (12 of 6,100, window 512: 2 % of the
// gradients' time).
template <int RB, bool KEYS>
__device__ inline Block find_block(const PromptArgs &a, int s, int mixed) {
    Block x;
    if (!a.cu) {
        const int per = (a.T + RB - 1) / RB, alone = (a.B - mixed) * per;
        const bool last = mixed > 0 && s >= alone;
        const int u = last ? s - alone : s, by = last ? mixed : per;
        const int hi = uniform(u / by), lo = u - hi * by;
        const int b = last ? a.B - mixed + lo : hi, r = last ? hi : lo;
        x.i = KEYS ? r : per - 1 - r;
        x.row0 = (KEYS ? b : a.B - 1 - b) * a.T;
        x.len = a.T;
        return x;
    }
    auto at = [&](int b) {
        const int c = a.cu[b];
        return c < 0 ? 0 : (c > a.T_total ? a.T_total : c);
    };
    const int lane = threadIdx.x & 63;
    if (mixed) {                             // (64 sequences at most, one a lane)
        const int row0 = lane < a.B ? at(lane) : 0, len = lane < a.B ? at(lane + 1) - row0 : 0;
        const int n = len > 0 ? (len - 1) / RB + 1 : 0;
        // blocks with at least t of their sequence on their shorter side
        auto longer = [&](int t) { return wave_sum(n > t ? n - t : 0); };
        int lo = 0, hi = a.T_total / RB + 1;          // longer(lo) > s, longer(hi) <= s
        x.i = -1;
        if (longer(0) <= s) return x;
        while (hi - lo > 1) {
            const int t = (lo + hi) / 2;
            if (longer(t) > s) lo = t;
            else               hi = t;
        }
        // (the sum by all lanes, ahead of what only some of them do)
        const int rank = s - longer(hi);
        const unsigned long long have = __builtin_amdgcn_ballot_w64(n > lo);
        const unsigned long long mine = __builtin_amdgcn_ballot_w64(
            (n > lo) & (__builtin_popcountll(have & ((1ull << lane) - 1)) == rank));
        if (!mine) return x;
        const int b = __builtin_ctzll(mine);
        x.i = KEYS ? __builtin_amdgcn_readlane(n, b) - 1 - lo : lo;
        x.row0 = __builtin_amdgcn_readlane(row0, b);
        x.len = __builtin_amdgcn_readlane(len, b);
        return x;
    }
    if (!KEYS) s = (int)((long long)a.T_total / RB + a.B) - 1 - s;
    int base = 0, count = a.B;               // the sequence is in [base, base + count)
    while (count > 1) {
        const int step = (count + 63) / 64, b = base + lane * step;
        const bool before = lane * step < count && at(b) / RB + b <= s;
        int last = __builtin_popcountll(__builtin_amdgcn_ballot_w64(before)) - 1;
        last = last < 0 ? 0 : last;
        base += last * step;
        count = count - last * step < step ? count - last * step : step;
    }
    const int lo = uniform(at(base)), hi = uniform(at(base + 1));
    x.i = s - (lo / RB + base);
    x.row0 = lo;
    x.len = hi - lo;
    if (x.i < 0 || x.len <= 0 || x.i > (x.len - 1) / RB) x.i = -1;
    return x;
}

// How many (of packed sequences only where they are 64 at most): in fp32 all, in bf16,
// whose products wait for what comes from beyond the caches, as many as keep the card's
// places for workgroups (`resident`) as long as the longest block takes, over h heads.
// Where a window is less than half of a sequence most blocks are as long, and bf16 calls
// go sequence by sequence.  In turn on warmed calls, us so, and sequence by sequence:
//   fp32, forward: 4 sequences of 4,096 tokens, 8 heads of 64, 577, 778 (packed: 579,
//     757), 8 of 1,000 to 4,096 548, 678, 8 of 700 to 2,900, 16 heads, window 1,024 424,
//     492, window 700 348, 384; gradients, 8 of 4,407, window 1,022, 2,187, 2,401; the
//     worst of 50 sizes 4 % slower (5 of 100 to 605, 64 heads of 128);
//   bf16, gradients of 12 x 1,024, 16 heads of 64 138, 145; forward, 9 of 400 to 2,356, 8
//     heads of 128 18 % sooner; all of 64 sequences of 1,024, 32 heads of 128 804, with
//     the last 4 737, with none 740; 17 of 1,517, window 446, 8 heads of 64 37 with all,
//     41 as it is, 38 of 649, window 207, 8 heads of 128 10 % slower with all.
template <typename T, int RB>
inline int mixed_seqs(const PromptArgs &a, int h, int resident) {
    if (a.cu && a.B > 64) return 0;
    if (sizeof(T) == 4) return a.B;
    const long long n = (a.cu ? a.T_total / a.B : a.T) / RB + 1, m = a.window > 0 ? a.window / RB + 1 : n;
    if (2 * m < n) return 0;
    const long long g = (2LL * resident + h * (n + 1) - 1) / (h * (n + 1));
    if (a.cu) return 2 * g < a.B ? 0 : a.B;
    return (int)(g < a.B ? g : a.B);
}

// Whether blocks of 32 rows (prompt_short.hip) are done sooner than blocks of 128.  The
// long form's time is that of its longest workgroups while it has few of them, the short
// form's, which spreads a block over four workgroups and reads every tile four times as
// often, that of all.  So what counts is the blocks of 32 times what a mean one attends
// to, as a share of the longest of 128, against a limit that grows with the longest loop
// (of the keys' kernel: times the heads of a group).  Its unit is 4 blocks of 128 half
// full, so that without a window it is the long form's workgroups; packed sequences,
// whose lengths differ, count for 7 / 8.
//   Measured, long against short, in us (the kernels alone; of the gradients both, the
// other one in the long form):
//   bf16, 128 channels: forward, 64 workgroups of 256 tokens 10.7 / 8.0, 128 10.6 / 13.1,
//     128 of 1,024 22.7 / 20.1, 192 22.9 / 29.4, of 4,096 73 / 68, 256 73 / 81;
//     queries, 192 of 2,048 127 / 115, 256 128 / 130; keys, 128 of 1,024 73 / 66, 192
//     74 / 84;
//   64 channels: forward, 128 of 512 10.2 / 7.7, 192 10.2 / 11.5, 256 of 2,048 28.2 /
//     24.7, 384 29.5 / 33.5; keys, 192 of 2,048 67.6 / 65.2, 256 69.2 / 72.5;
//   fp32, 64 channels: forward, 256 of 512 42.6 / 40.8, 384 55.7 / 65.1, 384 of 1,024
//     98.8 / 94.1, 512 106 / 122, of 2,048 204 / 201, 768 265 / 305; with a window of
//     1,024, 192 of 4,096 89.8 / 83.7, 256 89.2 / 102; keys, 384 of 2,048 574 / 565, 512
//     617 / 672, of 4 heads a group, 384 1,797 / 1,636, 512 2,085 / 2,159;
//   128 channels: forward, 256 of 512 78.1 / 72.9, 384 85.9 / 112, of 4,096 561 / 515,
//     512 605 / 672; keys, 256 of 1,024 499 / 424, 384 505 / 533, packed, of 512 to 2,048
//     tokens, 4 heads a group, 400 3,341 / 2,773, 650 4,473 / 4,546.
// Over 1,667 sizes of 50 to 4,800 tokens, windows and packed batches among them, the form
// taken is 0.2 % slower than the faster one in the mean, and past 10 % in 14 of 5,001 (up
// to 42 %, of 6 us: 8 of 174 tokens, window 31).
enum class Pass { kForward, kQueries, kKeys };
// of longest loops of fewer than 384, 1,024, 2,048, 4,096 tokens, and of more
struct Few { int blocks[5]; };
template <typename T, int D, Pass PASS>
constexpr Few few_blocks() {
    constexpr bool kWide = D == 128;
    if (sizeof(T) == 4) {
        if (PASS == Pass::kForward) return kWide ? Few{196, 316, 336, 416, 448} : Few{196, 300, 392, 576, 640};
        if (PASS == Pass::kQueries) return kWide ? Few{140, 316, 336, 388, 448} : Few{160, 238, 392, 576, 576};
        return kWide ? Few{164, 344, 376, 424, 448} : Few{208, 304, 400, 424, 544};
    }
    if (PASS == Pass::kForward) return kWide ? Few{65, 100, 136, 182, 224} : Few{100, 166, 250, 360, 360};
    if (PASS == Pass::kQueries) return kWide ? Few{65, 120, 208, 248, 288} : Few{72, 172, 312, 376, 440};
    return kWide ? Few{66, 120, 150, 176, 194} : Few{48, 110, 176, 240, 264};
}
template <typename T, int D, Pass PASS>
inline bool few_rows(const PromptArgs &a) {
    constexpr Few kFew = few_blocks<T, D, PASS>();
    const int h = PASS == Pass::kKeys ? a.Hkv : a.Hq;
    const long long len = a.T_total > a.B ? a.T_total / a.B : 1, w = a.window;
    const bool windowed = w > 0 && w < len;
    const long long blocks = (a.cu ? (a.T_total + 31LL) / 32 + a.B / 2 : a.B * ((len + 31) / 32)) * h;
    const long long top = windowed && w + 128 < len ? w + 128 : len;
    const long long mean = windowed ? 2 * w - w * w / len + 32 : len;      // (twice)
    const long long loop = PASS == Pass::kKeys ? top * a.G : top;
    const int step = (loop >= 384) + (loop >= 1024) + (loop >= 2048) + (loop >= 4096);
    // (mean / top is over 1 / 4, so that a call taken is far from filling a launch)
    return blocks * mean * (a.cu ? 7 : 8) <= 32 * top * kFew.blocks[step];
}

// The query head of workgroup number u of a block's Hq: workgroups go to the
// eight XCDs in turn, so that those which read one key-value head are a multiple
// of Hkv apart, on one XCD's L2 (or few).
__device__ inline int query_head(const PromptArgs &a, int u) { return u % a.Hkv * a.G + u / a.Hkv; }

// Rows of 32 tokens as MFMA operands, and products with tiles of rows that lie
// in LDS.  All three kernels are made of two products, with lane = 32 h + r:
//   rows:  X = tile . b^T, b 32 rows in registers: the lane gets X[j][r] for
//     the tile's rows j = key(e, h), value e of the accumulator;
//   cols:  acc^T += tile^T . P, P = 32 columns of which the lane holds
//     P[key(e, h)][r], e ascending: what `rows` gave, as it lies, the sum
//     running over the tile's rows in whatever order both operands use.  The
//     lane gets acc[c][e] = channel dim(c, e, h) of row r.
//
// A tile's rows are stored in chunks of 16 bytes, chunk c of row j at place
// c ^ swz(j): 16 lanes that read one chunk of 16 rows (`rows`) and 32 that
// read pieces of four rows (`cols`) then meet every bank once.
template <typename T, int D> struct Rows;

template <int D> struct Rows<bf16, D> {
    typedef bf16 T;
    static constexpr int kTok = 64, kRowBytes = 2 * D, kChunks = D / 8;
    static constexpr int kTileBytes = kTok * kRowBytes;
    static constexpr int kCols = D / 32;              // accumulators of `cols`
    struct B { bf16x8 f[D / 16]; };
    __device__ static inline int key(int e, int h) { return 8 * (e >> 2) + 4 * h + (e & 3); }
    __device__ static inline int dim(int c, int e, int h) { return D / 2 * h + 16 * c + e; }
    __device__ static inline int swz(int j) {
        if constexpr (D == 128) return ((j & 3) << 1) | ((j >> 2) & 1) | (((j >> 3) & 1) << 3);
        else return (((j >> 1) & 1) << 1) | ((j >> 2) & 1) | (((j >> 3) & 1) << 2);
    }
    // a number for each of a block's 32 rows, where `rows` has that row's
    __device__ static inline f32x16 per_row(const float *x, int h) {
        f32x16 y;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(x + key(e, h));
#pragma unroll
            for (int u = 0; u < 4; ++u) y[e + u] = v[u];
        }
        return y;
    }
    // row: the lane's row of b
    __device__ static inline void load(B &b, const T *row, int h) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) b.f[i] = ld8(row + 16 * i + 8 * h);
    }
    // makes the loads of b end here, not in a loop that follows
    __device__ static inline void settle(B &b) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(b.f[i]));
    }
    __device__ static inline void negate(B &b) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            b.f[i] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, b.f[i]) ^ 0x80008000u);
    }
    // what a lane adds to a tile's address in `rows` and in `cols`
    struct At { int row, col; };
    __device__ static inline At at(int lane) {
        const int r = lane & 31, h = lane >> 5, j = lane & 15;
        At a;
        a.row = r * kRowBytes + ((h ^ swz(r)) << 4);
        // lane j of 16 reads four channels of row 4 h + j / 4: of the segments
        // m / 4 = 4 (lane / 16 % 2) + j % 4 of the accumulator's rows m
        const int seg = 4 * ((lane >> 4) & 1) + (j & 3), row = 4 * h + (j >> 2);
        const int q = seg >> 1, chunk = D / 16 * (seg & 1) + (q >> 1);
        a.col = row * kRowBytes + ((chunk ^ swz(row)) << 4) + 8 * (q & 1);
        return a;
    }
    // rows 32 blk .. of the tile, the sums from s on
    __device__ static inline f32x16 rows(const char *tile, int blk, const At &a, const B &b,
                                         f32x16 s = f32x16{}) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const bf16x8 x = *reinterpret_cast<const bf16x8 *>(
                tile + 32 * blk * kRowBytes + (a.row ^ (i << 5)));
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, b.f[i], s, 0, 0, 0);
        }
        return s;
    }
    // After `rows` of N blocks: six of the reads from LDS go ahead of the products
    // that need them (16 packed prompts of 512 to 8,192 tokens, 32 heads over 8 of
    // 128: 1,722 us, 1,765 in the compiler's order).
    template <int N>
    __device__ static inline void ahead() {
        constexpr int kMfma = 0x8, kRead = 0x100, kAll = N * D / 16;
        __builtin_amdgcn_sched_group_barrier(kRead, 6, 0);
#pragma unroll
        for (int i = 0; i < kAll - 6; ++i) {
            __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, 6, 0);
    }
    // Weights (and their gradients) as one bf16 number each, off by at most 2^-8:
    // with two, as in the attention of new tokens, where bytes bound the call, a
    // forward call of the sizes above takes 2,459 us for 1,822, and o's error
    // against 64 bits is 1.65e-3 (that of rounding o itself) for 2.17e-3.
    struct P { bf16x8 f[2]; };
    __device__ static inline P operand(const f32x16 &x) {
        P p;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int u = 0; u < 8; ++u) p.f[k][u] = (bf16)x[8 * k + u];
        return p;
    }
    // Weights as the sum of two bf16 numbers: hi, cut to bf16, and lo, the rest
    // rounded to it, off by at most 2^-15 of a weight together.  The rest gains
    // 2^-23 of the weight, so that lo is above 0 where the weight is and an
    // infinity that a row attends to meets no 0.
    struct Two { P hi, lo; };
    __device__ static inline Two operand2(const f32x16 &x) {
        Two p;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            u32x4 hi;
            float lo[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float a = x[8 * k + 2 * u], b = x[8 * k + 2 * u + 1];
                const unsigned ab = __builtin_bit_cast(unsigned, a), bb = __builtin_bit_cast(unsigned, b);
                hi[u] = __builtin_amdgcn_perm(bb, ab, 0x07060302u);
                lo[2 * u] = fmaf(a, 1.f + 0x1p-23f, -__builtin_bit_cast(float, ab & 0xFFFF0000u));
                lo[2 * u + 1] = fmaf(b, 1.f + 0x1p-23f, -__builtin_bit_cast(float, bb & 0xFFFF0000u));
            }
            p.hi.f[k] = __builtin_bit_cast(bf16x8, hi);
            p.lo.f[k] = cvt8(lo);
        }
        return p;
    }
    // rows 32 blk + 16 k .. as the operand of channel block c
    __device__ static inline bf16x8 col_frag(const char *tile, int blk, int k, int c, const At &a) {
        const char *t = tile + (32 * blk + 16 * k) * kRowBytes;
        const int flip = swz(8) << 4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(t + (a.col ^ (c << 5))));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(t + 8 * kRowBytes + (a.col ^ (c << 5) ^ flip)));
        return cat8(__builtin_bit_cast(bf16x4, lo), __builtin_bit_cast(bf16x4, hi));
    }
    // without infinities and NaN (an exponent of all ones)
    __device__ static inline bf16x8 clear(bf16x8 x) {
        u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = ((w[i] & 0x7F80u) == 0x7F80u ? 0u : w[i] & 0xFFFFu) |
                   ((w[i] & 0x7F800000u) == 0x7F800000u ? 0u : w[i] & 0xFFFF0000u);
        return __builtin_bit_cast(bf16x8, w);
    }
    // CLEAR: without the tile's infinities and NaN, unless all of it counts
    template <bool CLEAR>
    __device__ static inline void cols(f32x16 (&acc)[kCols], const char *tile, int blk, const At &a,
                                       const P &p, bool all) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                bf16x8 x = col_frag(tile, blk, k, c, a);
                if constexpr (CLEAR) x = all ? x : clear(x);
                acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, p.f[k], acc[c], 0, 0, 0);
            }
    }
    template <bool CLEAR>
    __device__ static inline void cols(f32x16 (&acc)[kCols], const char *tile, int blk, const At &a,
                                       const Two &p, bool all) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                bf16x8 x = col_frag(tile, blk, k, c, a);
                if constexpr (CLEAR) x = all ? x : clear(x);
                acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, p.hi.f[k], acc[c], 0, 0, 0);
                acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, p.lo.f[k], acc[c], 0, 0, 0);
            }
    }
    __device__ static inline bool any_odd(const f32x16 (&acc)[kCols]) {
        bool y = false;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) y |= !(fabsf(acc[c][e]) < INFINITY);
        return y;
    }
    // adds a row's infinities and NaN
    __device__ static inline void add_odd(f32x16 (&acc)[kCols], const T *row, int h) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = (float)row[dim(c, e, h)];
                acc[c][e] += fabsf(x) < INFINITY ? 0.f : x;
            }
    }
    // a row's accumulators into D floats
    __device__ static inline void put(float *row, const f32x16 (&acc)[kCols], int h) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<f32x4 *>(row + dim(c, e, h)) =
                    f32x4{acc[c][e], acc[c][e + 1], acc[c][e + 2], acc[c][e + 3]};
    }
    // acc[.][.] of one row: D / 2 channels from D / 2 h on
    __device__ static inline void store(T *row, const f32x16 (&acc)[kCols], int h, float f) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float y[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) y[u] = acc[c][8 * k + u] * f;
                *reinterpret_cast<bf16x8 *>(row + dim(c, 8 * k, h)) = cvt8(y);
            }
    }
};

template <int D> struct Rows<float, D> {
    typedef float T;
    static constexpr int kTok = 32, kRowBytes = 4 * D, kChunks = D / 4;
    static constexpr int kTileBytes = kTok * kRowBytes;
    static constexpr int kCols = D / 32;
    struct B { f32x4 f[D / 8]; };
    __device__ static inline int key(int e, int h) { return 8 * (e >> 2) + 4 * h + (e & 3); }
    __device__ static inline int dim(int c, int e, int h) { return kCols * key(e, h) + c; }
    __device__ static inline int swz(int j) { return j & 15; }
    // a number for each of a block's 32 rows, where `rows` has that row's
    __device__ static inline f32x16 per_row(const float *x, int h) {
        f32x16 y;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(x + key(e, h));
#pragma unroll
            for (int u = 0; u < 4; ++u) y[e + u] = v[u];
        }
        return y;
    }
    __device__ static inline void load(B &b, const T *row, int h) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) b.f[i] = *reinterpret_cast<const f32x4 *>(row + 8 * i + 4 * h);
    }
    // makes the loads of b end here, not in a loop that follows
    __device__ static inline void settle(B &b) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) asm volatile("" : "+v"(b.f[i]));
    }
    __device__ static inline void negate(B &b) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) b.f[i] = -b.f[i];
    }
    struct At { int row, col; };
    __device__ static inline At at(int lane) {
        const int r = lane & 31, h = lane >> 5, byte = 4 * kCols * r;
        At a;
        a.row = r * kRowBytes + ((h ^ swz(r)) << 4);
        a.col = 4 * h * kRowBytes + (((byte >> 4) ^ swz(4 * h)) << 4) + (byte & 15);
        return a;
    }
    __device__ static inline f32x16 mfma(float a, float b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
    }
    // two sums of D / 2 products, then theirs
    __device__ static inline f32x16 rows(const char *tile, int blk, const At &a, const B &b,
                                         f32x16 s = f32x16{}) {
        f32x16 t{};
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(
                tile + 32 * blk * kRowBytes + (a.row ^ (i << 5)));
            s = mfma(x[0], b.f[i][0], s);
            t = mfma(x[1], b.f[i][1], t);
            s = mfma(x[2], b.f[i][2], s);
            t = mfma(x[3], b.f[i][3], t);
        }
        return s + t;
    }
    template <int N> __device__ static inline void ahead() {}
    struct P { f32x16 f; };
    __device__ static inline P operand(const f32x16 &x) { return P{x}; }
    typedef float run_t __attribute__((ext_vector_type(kCols)));
    // row key(e, h) of block blk: channels kCols r ..
    __device__ static inline run_t col_frag(const char *tile, int blk, int e, const At &a) {
        const int j = 8 * (e >> 2) + (e & 3);
        return *reinterpret_cast<const run_t *>(tile + (32 * blk + j) * kRowBytes +
                                                (a.col ^ (swz(j) << 4)));
    }
    // (a value parameter: the bit cast of a vector's element in place takes the
    // vector's first element)
    __device__ static inline unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }
    __device__ static inline bool odd(float x) { return (bits(x) & 0x7F800000u) == 0x7F800000u; }
    template <bool CLEAR>
    __device__ static inline void cols(f32x16 (&acc)[kCols], const char *tile, int blk, const At &a,
                                       const P &p, bool all) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const run_t x = col_frag(tile, blk, e, a);
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[c] = mfma(CLEAR && !all && odd(x[c]) ? 0.f : x[c], p.f[e], acc[c]);
        }
    }
    __device__ static inline bool any_odd(const f32x16 (&acc)[kCols]) {
        bool y = false;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) y |= !(fabsf(acc[c][e]) < INFINITY);
        return y;
    }
    __device__ static inline void add_odd(f32x16 (&acc)[kCols], const T *row, int h) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = row[dim(c, e, h)];
                acc[c][e] += odd(x) ? x : 0.f;
            }
    }
    __device__ static inline void put(float *row, const f32x16 (&acc)[kCols], int h) {
        store(row, acc, h, 1.f);
    }
    __device__ static inline void store(T *row, const f32x16 (&acc)[kCols], int h, float f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            run_t y;
#pragma unroll
            for (int c = 0; c < kCols; ++c) y[c] = acc[c][e] * f;
            *reinterpret_cast<run_t *>(row + dim(0, e, h)) = y;
        }
    }
};

// Sums of weights times values are divided by the weights' sum only at the end, so that
// finite values of V may sum to infinities.  Rows where they did are summed again with
// weights times kDown: those are then at most 2^-30 (2^8 where a maximum is left
// behind), and the sums of fewer than 2^29 tokens below the largest value.
constexpr float kDown = 0x1p-38f, kUp = 0x1p38f;
// One bit for each of the wave's 32 rows: whether `odd` is set in either half.
__device__ inline unsigned rows_of(bool odd) {
    const unsigned long long m = __builtin_amdgcn_ballot_w64(odd);
    return (unsigned)m | (unsigned)(m >> 32);
}

// What the backward pass keeps of a row in its workspace: lse log2 e (+inf for a
// row without weights) and -delta = -do . o, from which the sums do . v start, of
// which each half of a wave sums half the channels.
__device__ inline float base2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }
template <typename T, int D>
__device__ inline float minus_delta(const T *d_o, const T *o, int h) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 2; i += 8) {
#pragma unroll
        for (int u = 0; u < 8; u += 4) {
            const f32x4 x = Elem<T>::load4(d_o + D / 2 * h + i + u);
            const f32x4 y = Elem<T>::load4(o + D / 2 * h + i + u);
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fmaf(-x[e], y[e], s);
        }
    }
    return swap_sum32(s);
}

// Loads straight from memory into LDS, 16 bytes a lane, in the lanes' order.
// (Written out: the compiler would wait for a load to LDS before the next read
// of any LDS.)
__device__ inline unsigned lds_address(const char *p) {
    return (unsigned)reinterpret_cast<size_t>((const lds_void *)p);
}
// memory from `from` on; what lies at `bytes` and past it comes as zeros
__device__ inline u32x4 source(const char *from, unsigned bytes) {
    const unsigned long long base = reinterpret_cast<unsigned long long>(from);
    return u32x4{(unsigned)uniform((int)base), (unsigned)uniform((int)(base >> 32)),
                 (unsigned)uniform((int)bytes), 0x00020000u};
}
__device__ inline void load_lds(unsigned to, u32x4 from, unsigned off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(uniform((int)to)), "v"(off), "s"(from) : "memory");
}

// Rows row0 .. of a head ([rows, heads, D], heads * D elements apart) into a
// tile in LDS, by the waves of a workgroup, straight from memory: a wave's
// instruction fills 1 KiB, 16 bytes a lane in their order, so that the lane
// asks for the chunk that belongs there.  Rows from `valid` (>= 1) on are
// copies of the last one, which the callers mask.  What a lane adds to a tile's
// address is the same for all whole tiles.
template <typename T, int D, int WAVES>
struct Fetch {
    using R = Rows<T, D>;
    static constexpr int kPer = 1024 / R::kRowBytes, kLoads = R::kTok / kPer / WAVES;
    static_assert(kLoads * kPer * WAVES == R::kTok, "the waves fetch alike");
    unsigned pitch, off[kLoads];
    int w;
    __device__ static inline int row(int i, int w, int lane) {
        return (w + WAVES * i) * kPer + lane / R::kChunks;
    }
    __device__ static inline unsigned chunk(int row, int lane) {
        return 16u * (lane % R::kChunks ^ R::swz(row));
    }
    __device__ inline Fetch(unsigned pitch, int w, int lane) : pitch(pitch), w(w) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int j = row(i, w, lane);
            off[i] = j * pitch + chunk(j, lane);
        }
    }
    __device__ inline void operator()(char *tile, const T *head, size_t row0, int valid,
                                      int lane) const {
        const u32x4 from = source(reinterpret_cast<const char *>(head) + row0 * pitch, 0xFFFFFFFFu);
        const unsigned to = lds_address(tile) + 1024u * w;
        if (valid >= R::kTok) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load_lds(to + 1024u * WAVES * i, from, off[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int j = row(i, w, lane), last = j < valid ? j : valid - 1;
                load_lds(to + 1024u * WAVES * i, from, last * pitch + chunk(j, lane));
            }
        }
    }
};
// 4 bytes a lane of `from` (its element `index`), lanes 0 .. N - 1, into words
// that lie together in LDS, likewise.
template <int N>
__device__ inline void fetch_words(float *to, const float *from, int index, int lane) {
    const u32x4 rs = source(reinterpret_cast<const char *>(from), 0xFFFFFFFFu);
    const int at = uniform((int)lds_address(reinterpret_cast<const char *>(to)));
    if (lane < N)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     :: "s"(at), "v"(4u * index), "s"(rs) : "memory");
}
// After fetch: waits until every wave's part is there, and until every wave is
// done with what it read before.
__device__ inline void tile_landed() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

}  // namespace gdr

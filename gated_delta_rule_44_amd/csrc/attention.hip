// attention.hip -- attention of new tokens over the paged key-value cache,
// for gfx950.
//
// Row (b, t, h) of the queries stands at position p = len_b - n + t and
// attends to the cached tokens j <= p (and j > p - window):
//     s_j = scale q.k_j,   w_j = e^{s_j} / sum e^{s_i},   o = sum w_j v_j.
//
// One pass over K and V with a running maximum m and sum l (in units of
// log2: x = s log2 e): for a tile of tokens, m' = max(m, max x),
// l = l 2^{m - m'} + sum 2^{x - m'}, o likewise.  Parts of a sequence join by
// the same rule.
//
// The G = Hq / Hkv query heads of a key-value head and the n new tokens make
// n G rows that read the same K and V: 16 R rows are one workgroup's, so
// that a token is read from HBM once for all of them, as MFMA operands.
// Bytes bound the kernel: 2 D elements a token against 4 D flops per row and
// token is at most 16 R flops a byte, where the card turns at about 250.
#include "cache_internal.h"
#include "gdr_internal.h"
#include "device_util.h"

namespace gdr {
namespace {

constexpr int kWaves = 4;                  // waves of a workgroup
constexpr int kThreads = 64 * kWaves;

// First and one past the last token that query token t of a sequence of len
// tokens attends to (empty when lo >= hi).
struct Span { int lo, hi; };
__device__ inline Span token_span(int len, int n, int window, int t) {
    const int p = len - n + t;
    return Span{window > 0 && p >= window ? p - window + 1 : 0, p + 1};
}
// The tokens that any row of a sequence attends to, from a multiple of 32.
__device__ inline Span seq_span(int len, int n, int window) {
    const int lo = token_span(len, n, window, 0).lo;
    return Span{lo & ~31, len};
}

// How the cached tokens are shared out.  Every sequence's span is cut into
// chunks of C tokens, the same C for all, so that a long sequence among short
// ones is spread over as many workgroups as its length asks for; C follows
// from the lengths on the device, such that about kTargetWgs workgroups
// have work.  Chunks are numbered over the sequences ("slots"); a sequence
// without tokens has one, which writes its zeros.
constexpr int kTargetWgs = 1024;
constexpr int kMinChunk = 512;
struct Plan {
    int units;            // workgroups of one slot: key-value heads x row blocks
    int row_blocks;       // blocks of 16 R rows
    int want_slots;       // slots aimed at
    int max_slots;        // bound on the slots there can be: sum ceil(len / C) <= want + B
};
Plan make_plan(int B, int n, int G, int Hkv, int R, long long capacity) {
    Plan p;
    p.row_blocks = (n * G + 16 * R - 1) / (16 * R);
    p.units = Hkv * p.row_blocks;
    p.want_slots = p.units >= kTargetWgs ? 1 : kTargetWgs / p.units;
    const long long by_len = (capacity + kMinChunk - 1) / kMinChunk * B;
    const long long bound = (long long)p.want_slots + B;
    p.max_slots = (int)(by_len < bound ? (by_len < B ? B : by_len) : bound);
    return p;
}
// Rows of a workgroup's block, in tiles of 16, one per wave: the four waves
// are R tiles of rows x 4 / R shares of the tokens.  Waves of one share read
// the same K and V, from HBM once and then from the CU's L1.
int row_tiles(long long rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

// Workspace: {first slot, slots} of every sequence; (m, l) of every slot, unit
// and row; o of the same, unnormalised; with scores, the logits x of every row and
// token [B, Hkv, nG, cap].
struct WsMap {
    size_t sched, ml, o, logits, total;
};
WsMap ws_map(int B, int n, int G, int Hkv, int D, int R, long long capacity, bool with_scores) {
    auto r256 = [](size_t x) { return (x + 255) / 256 * 256; };
    const Plan p = make_plan(B, n, G, Hkv, R, capacity);
    const size_t rows = (size_t)p.max_slots * p.units * 16 * R;
    const bool parts = p.max_slots > B;
    WsMap w{};
    w.sched = 0;
    w.ml = r256((size_t)B * 2 * sizeof(int));
    w.o = w.ml + (parts || with_scores ? r256(rows * 2 * sizeof(float)) : 0);
    w.logits = w.o + (parts ? r256(rows * D * sizeof(float)) : 0);
    w.total = w.logits + (with_scores ? (size_t)B * Hkv * n * G * ((capacity + 31) / 32 * 32) *
                                            sizeof(float) : 0);
    return w;
}

struct KArgs {
    AttnArgs a;
    Plan plan;
    int2 *sched;
    float2 *ml;
    float *po;
    float *logits;        // nullptr: no scores
    long long cap32;      // tokens of a logits row
    bool parts;           // a sequence may have several slots
};

// Sum over the workgroup's threads before this one and over all; lds holds
// kWaves values.
template <typename N>
__device__ inline N group_scan(N x, N &total, N *lds) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    N incl = x;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const N y = __shfl_up(incl, m);
        if (lane >= m) incl += y;
    }
    if (lane == 63) lds[w] = incl;
    __syncthreads();
    N before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const N v = lds[i];
        before += i < w ? v : 0;
        total += v;
    }
    __syncthreads();
    return before + incl - x;
}

struct Slot { int b, first, count, chunk; };      // sequence, its first slot, its slots, C
// The sequence that slot s belongs to (b = -1: past the last slot).  Thread
// i of the workgroup looks after sequences i per .. i per + per - 1.
__device__ inline Slot find_slot(const KArgs &k, int s) {
    // too short a table for a second slot: slot and sequence are one
    if (!k.parts) return Slot{s < k.a.B ? s : -1, s, 1, 1 << 30};
    __shared__ long long lds64[kWaves];
    __shared__ int lds32[kWaves], found[3];
    const AttnArgs &a = k.a;
    const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
    long long sum = 0, total;
    for (int b = b0; b < b0 + per && b < a.B; ++b) {
        const Span sp = seq_span(cached_len(a.seq_lens, b, a.map), a.n, a.window);
        sum += sp.hi - sp.lo;
    }
    group_scan<long long>(sum, total, lds64);
    long long c = (total + k.plan.want_slots - 1) / k.plan.want_slots;
    c = c < kMinChunk ? kMinChunk : (c > (1 << 30) ? 1 << 30 : c);
    const int chunk = (int)((c + 127) / 128 * 128);
    int mine = 0, slots;
    for (int b = b0; b < b0 + per && b < a.B; ++b) {
        const Span sp = seq_span(cached_len(a.seq_lens, b, a.map), a.n, a.window);
        const int ns = (sp.hi - sp.lo + chunk - 1) / chunk;
        mine += ns > 1 ? ns : 1;
    }
    if (threadIdx.x == 0) found[0] = -1;
    int at = group_scan<int>(mine, slots, lds32);
    if (s >= at && s < at + mine) {
        for (int b = b0; b < b0 + per && b < a.B; ++b) {
            const Span sp = seq_span(cached_len(a.seq_lens, b, a.map), a.n, a.window);
            int ns = (sp.hi - sp.lo + chunk - 1) / chunk;
            ns = ns > 1 ? ns : 1;
            if (s < at + ns) {
                found[0] = b; found[1] = at; found[2] = ns;
                break;
            }
            at += ns;
        }
    }
    __syncthreads();
    return Slot{found[0], found[1], found[2], chunk};
}

__device__ inline float swap_max16(float x) {
    float a = x, b = x;
    asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(b));
    return fmaxf(a, b);
}
__device__ inline float swap_max32(float x) {
    float a = x, b = x;
    asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
    return fmaxf(a, b);
}
__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
// What logits are taken relative to: their maximum, or 0 where every one is
// -inf (masked, then the weights 2^{-inf} are 0) or NaN (which fmaxf passes
// over and the weights keep).
__device__ inline float finite_top(float m) { return m == -INFINITY ? 0.f : m; }

// K and V are read once by one wave (R = 1): loads that pass through the
// caches without staying there (64 contexts, 680 MB: 142 -> 129 us).
constexpr int kStream = 2;
__device__ inline u32x4 stream16(rsrc_t r, unsigned off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kStream);
}

// A tile's operands, per dtype.  With lane = 16 lg + r:
//   S^T = K Q^T: lane supplies key r of a block of 16 (A) and query row r (B),
//     and gets the logits of query row r with keys 4 lg .. 4 lg + 3;
//   O^T = V^T P^T: P^T's operand is those logits' weights as they lie (the
//     sum over k runs over the keys in whatever order both operands use),
//     and V^T's is read from rows 4 lg + e of V, PER = D / 16 channels per
//     lane, so that V needs no transposition through LDS: acc[c][e] is
//     channel dim(c, 4 lg + e) of query row r.
// Several waves that read one tile (R > 1) take it from LDS, where it lies row
// by row, the 16-byte chunks of a row exchanged by its number (chunk c at
// c ^ swap(row)), so that the sixteen rows of a K operand are in different
// banks.
template <typename T, int D> struct Tile;
template <int ROW_BYTES>
__device__ inline int chunk_at(int row, int c) {
    const int swap = ROW_BYTES >= 256 ? row & 15 : (row >> 1) & 7;
    return row * ROW_BYTES + ((c ^ swap) << 4);
}

template <int D> struct Tile<bf16, D> {
    static constexpr int kBlocks = 2;              // blocks of 16 tokens: 32 k slots
    static constexpr int PER = D / 16;
    static constexpr int kRowBytes = D * 2;
    struct Q { bf16x8 f[D / 32]; };
    struct K { bf16x8 f[2][D / 32]; };
    struct V { unsigned w[2][4][PER / 2]; };
    __device__ static inline int dim(int c, int m) { return PER * m + c; }
    __device__ static inline void load_q(Q &q, rsrc_t r, unsigned off, int lane) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) q.f[i] = bload16(r, off + 64 * i + 16 * (lane >> 4));
    }
    __device__ static inline void load_k(K &k, int blk, rsrc_t r, int lane) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            k.f[blk][i] = __builtin_bit_cast(
                bf16x8, stream16(r, (lane & 15) * kRowBytes + 64 * i + 16 * (lane >> 4)));
    }
    __device__ static inline void load_v(V &v, int blk, rsrc_t r, int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned off = (4 * (lane >> 4) + e) * kRowBytes + (lane & 15) * PER * 2;
            if constexpr (PER == 8) {
                const u32x4 x = stream16(r, off);
#pragma unroll
                for (int i = 0; i < 4; ++i) v.w[blk][e][i] = x[i];
            } else {
                const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, kStream);
                v.w[blk][e][0] = x[0];
                v.w[blk][e][1] = x[1];
            }
        }
    }
    __device__ static inline void lds_k(K &k, int blk, const char *t, int lane) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            k.f[blk][i] = *reinterpret_cast<const bf16x8 *>(
                t + chunk_at<kRowBytes>(16 * blk + (lane & 15), 4 * i + (lane >> 4)));
    }
    __device__ static inline void lds_v(V &v, int blk, const char *t, int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 16 * blk + 4 * (lane >> 4) + e, r = lane & 15;
            if constexpr (PER == 8) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(t + chunk_at<kRowBytes>(row, r));
#pragma unroll
                for (int i = 0; i < 4; ++i) v.w[blk][e][i] = x[i];
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(
                    t + chunk_at<kRowBytes>(row, r >> 1) + 8 * (r & 1));
                v.w[blk][e][0] = x.x;
                v.w[blk][e][1] = x.y;
            }
        }
    }
    __device__ static inline f32x4 logits(const K &k, int blk, const Q &q) {
        f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s = mfma32(k.f[blk][i], q.f[i], s);
        return s;
    }
    // weights rounded to bf16, as the product's operand must be: each is off
    // by at most 2^-8 of itself, and the signs of these errors average out
    // over a row's tokens; o itself is rounded to bf16 at the end
    struct P { bf16x8 f; };
    __device__ static inline P weights(const f32x4 *p) { return P{acc_pair(p[0], p[1])}; }
    __device__ static inline bf16x8 v_frag(const V &v, int c) {
        const unsigned sel = c & 1 ? 0x07060302u : 0x05040100u;
        u32x4 x;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                x[2 * blk + u] = __builtin_amdgcn_perm(v.w[blk][2 * u + 1][c >> 1],
                                                       v.w[blk][2 * u][c >> 1], sel);
        return __builtin_bit_cast(bf16x8, x);
    }
    __device__ static inline f32x4 pv(const V &v, int c, const P &p, f32x4 acc) {
        return mfma32(v_frag(v, c), p.f, acc);
    }
    // an infinity or NaN among this lane's values
    __device__ static inline bool odd(const V &v) {
        bool y = false;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < PER / 2; ++i)
                    y |= (v.w[blk][e][i] & 0x7F80u) == 0x7F80u ||
                         (v.w[blk][e][i] & 0x7F800000u) == 0x7F800000u;
        return y;
    }
    // 1 where a value is an infinity or NaN other than `but` (an infinity's
    // bits), times the 0 or 1 of ones, summed over the tile's tokens
    __device__ static inline f32x4 count_odd(const V &v, int c, unsigned but, const P &ones) {
        u32x4 x = __builtin_bit_cast(u32x4, v_frag(v, c));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned lo = x[i] & 0xFFFFu, hi = x[i] >> 16;
            x[i] = ((lo & 0x7F80u) == 0x7F80u && lo != but ? 0x3F80u : 0u) |
                   ((hi & 0x7F80u) == 0x7F80u && hi != but ? 0x3F800000u : 0u);
        }
        return mfma32z(__builtin_bit_cast(bf16x8, x), ones.f);
    }
    static constexpr unsigned kPlusInf = 0x7F80u, kMinusInf = 0xFF80u;
    __device__ static inline void clear_odd(V &v) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) {
                    const unsigned x = v.w[blk][e][i];
                    v.w[blk][e][i] = ((x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) |
                                     ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u);
                }
    }
};

template <int D> struct Tile<float, D> {
    static constexpr int kBlocks = 1;
    static constexpr int PER = D / 16;
    static constexpr int kRowBytes = D * 4;
    struct Q { f32x4 f[D / 16]; };
    struct K { f32x4 f[1][D / 16]; };
    struct V { f32x4 f[4][PER / 4]; };
    // a value parameter: the bit cast of a vector's element in place takes
    // the vector's first element
    __device__ static inline unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }
    // channels 64 (c / 4) + 4 m + c % 4: a load covers 256 bytes of a row
    __device__ static inline int dim(int c, int m) { return 64 * (c >> 2) + 4 * m + (c & 3); }
    __device__ static inline void load_q(Q &q, rsrc_t r, unsigned off, int lane) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) q.f[i] = bload16f(r, off + 64 * i + 16 * (lane >> 4));
    }
    __device__ static inline void load_k(K &k, int, rsrc_t r, int lane) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            k.f[0][i] = __builtin_bit_cast(
                f32x4, stream16(r, (lane & 15) * kRowBytes + 64 * i + 16 * (lane >> 4)));
    }
    __device__ static inline void load_v(V &v, int, rsrc_t r, int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                v.f[e][i] = __builtin_bit_cast(
                    f32x4, stream16(r, (4 * (lane >> 4) + e) * kRowBytes + 256 * i +
                                           16 * (lane & 15)));
    }
    __device__ static inline void lds_k(K &k, int, const char *t, int lane) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            k.f[0][i] = *reinterpret_cast<const f32x4 *>(
                t + chunk_at<kRowBytes>(lane & 15, 4 * i + (lane >> 4)));
    }
    __device__ static inline void lds_v(V &v, int, const char *t, int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                v.f[e][i] = *reinterpret_cast<const f32x4 *>(
                    t + chunk_at<kRowBytes>(4 * (lane >> 4) + e, 16 * i + (lane & 15)));
    }
    __device__ static inline f32x4 logits(const K &k, int, const Q &q) {
        f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s = __builtin_amdgcn_mfma_f32_16x16x4f32(k.f[0][i][e], q.f[i][e], s, 0, 0, 0);
        return s;
    }
    struct P { f32x4 f; };
    __device__ static inline P weights(const f32x4 *p) { return P{p[0]}; }
    __device__ static inline f32x4 pv(const V &v, int c, const P &p, f32x4 acc) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(v.f[e][c >> 2][c & 3], p.f[e], acc, 0, 0, 0);
        return acc;
    }
    __device__ static inline bool odd(const V &v) {
        bool y = false;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y |= (bits(v.f[e][i][j]) & 0x7F800000u) == 0x7F800000u;
        return y;
    }
    __device__ static inline f32x4 count_odd(const V &v, int c, unsigned but, const P &ones) {
        f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned u = bits(v.f[e][c >> 2][c & 3]);
            const float x = (u & 0x7F800000u) == 0x7F800000u && u != but ? 1.f : 0.f;
            s = __builtin_amdgcn_mfma_f32_16x16x4f32(x, ones.f[e], s, 0, 0, 0);
        }
        return s;
    }
    static constexpr unsigned kPlusInf = 0x7F800000u, kMinusInf = 0xFF800000u;
    __device__ static inline void clear_odd(V &v) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned u = bits(v.f[e][i][j]);
                    v.f[e][i][j] = (u & 0x7F800000u) == 0x7F800000u ? 0.f : v.f[e][i][j];
                }
    }
};

// Workgroup = (slot, key-value head, row block).  Wave w has row tile w % R
// and takes every 4 / R-th tile of tokens, with m, l and o of its own, joined
// through LDS at the end.
//
// R = 1: K and V go from HBM straight into the registers that MFMA reads: the
// next tile to come is requested into a tile's registers as they fall free, K
// after its logits are formed, V after its product.
// R > 1: the waves of a share read the same tiles, which all threads bring
// into LDS together, a stage (one tile per share) at a time: one stage is
// worked on, the next is written beside it, and two more are on the way in
// registers.
template <typename T, int D, int R>
__global__ __launch_bounds__(kThreads, 2) void attn_kernel(KArgs k) {
    using TL = Tile<T, D>;
    constexpr int PER = TL::PER, kBlocks = TL::kBlocks, kTile = 16 * kBlocks;
    constexpr int kPad = D + 4, kShares = kWaves / R;
    constexpr int kTileBytes = kTile * TL::kRowBytes, kStage = kShares * 2 * kTileBytes;
    constexpr int kOBytes = kWaves * 16 * kPad * (int)sizeof(float);
    __shared__ float sm[kWaves][16], sl[kWaves][16];
    // the stages, and at the end every wave's o
    __shared__ __align__(16) char lds[R > 1 && 2 * kStage > kOBytes ? 2 * kStage : kOBytes];
    float(*so)[16][kPad] = reinterpret_cast<float(*)[16][kPad]>(lds);
    const AttnArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), rt = w % R, share = w / R;
    // the row blocks of one (slot, head) follow each other on one XCD, which
    // holds their K and V in its L2 (workgroups go to the eight XCDs in turn)
    const int wg = blockIdx.x;
    const int rb = wg / 8 % k.plan.row_blocks;
    const int unit = wg / 8 / k.plan.row_blocks * 8 + wg % 8;
    const int slot = unit / a.Hkv, h = unit % a.Hkv;
    const Slot sl_ = find_slot(k, slot);
    const int b = sl_.b;
    if (b < 0) return;
    const int len = cached_len(a.seq_lens, b, a.map);
    const Span seq = seq_span(len, a.n, a.window);
    if (h == 0 && rb == 0 && slot == sl_.first && tid == 0) k.sched[b] = int2{sl_.first, sl_.count};

    // this lane's query row and what it attends to
    const int rows = a.n * a.G, row0 = rb * 16 * R, row = row0 + 16 * rt + r16;
    Span sp{0, 0};
    typename TL::Q q;
    {
        const size_t qb = (size_t)b * a.n * a.Hq * D;
        const rsrc_t rq = make_rsrc(static_cast<const T *>(a.q) + qb, 0xFFFFFFFFu);
        const int t = row < rows ? row / a.G : 0, g = row < rows ? row % a.G : 0;
        if (row < rows) sp = token_span(len, a.n, a.window, t);
        TL::load_q(q, rq, (unsigned)(t * a.Hq + h * a.G + g) * (D * (unsigned)sizeof(T)), lane);
    }
    // the block's tokens: what its rows attend to, within the slot
    const int t_first = row0 / a.G;
    const int t_last = ((row0 + 16 * R < rows ? row0 + 16 * R : rows) - 1) / a.G;
    const Span first = token_span(len, a.n, a.window, t_first);
    const Span last = token_span(len, a.n, a.window, t_last);
    const int c_lo = seq.lo + (slot - sl_.first) * sl_.chunk;
    const int c_hi = c_lo + sl_.chunk < len ? c_lo + sl_.chunk : len;
    const int k_lo = first.lo > c_lo ? first.lo : c_lo, k_hi = last.hi < c_hi ? last.hi : c_hi;
    // every row attends to the tokens of [all_lo, all_hi)
    const int all_lo = last.lo, all_hi = first.hi;
    const int tile0 = k_lo / kTile;
    const int tiles = k_hi > k_lo ? (k_hi + kTile - 1) / kTile - tile0 : 0;

    const char *kc = static_cast<const char *>(a.k_cache), *vc = static_cast<const char *>(a.v_cache);
    const float c1 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    f32x4 acc[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};

    // One tile's logits (before scaling) and values into m, l and o.  full:
    // every row attends to all of it; here: which of its blocks are there.
    auto absorb = [&](int j0, f32x4 (&x)[kBlocks], typename TL::V &vf, bool full,
                      const bool (&here)[kBlocks]) {
        float top = -INFINITY;
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[blk][e] *= c1;
            if (k.logits && row < rows && here[blk])
                *reinterpret_cast<f32x4 *>(k.logits +
                                           (((size_t)b * a.Hkv + h) * rows + row) * k.cap32 + j0 +
                                           16 * blk + 4 * lg) = x[blk];
            if (!full) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + 16 * blk + 4 * lg + e;
                    x[blk][e] = here[blk] && j >= sp.lo && j < sp.hi ? x[blk][e] : -INFINITY;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, x[blk][e]);
        }
        const float mn = fmaxf(m, swap_max32(swap_max16(top))), ms = finite_top(mn);
        if (__builtin_amdgcn_ballot_w64(mn != m)) {
            const float al = exp2_(m - ms);
            l *= al;
#pragma unroll
            for (int c = 0; c < PER; ++c) acc[c] *= al;
            m = mn;
        }
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[blk][e] = exp2_(x[blk][e] - ms);
                l += x[blk][e];
            }
        const typename TL::P p = TL::weights(x);
        // Where a tile is attended to by some rows only, a weight of zero must
        // not meet an infinity or NaN.  Such values are taken out of V, and a
        // row that attends to one gets +inf, -inf or (both, or NaN) their
        // sum in that channel.
        if (!full && __builtin_amdgcn_ballot_w64(TL::odd(vf))) {
            f32x4 in[kBlocks];
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + 16 * blk + 4 * lg + e;
                    in[blk][e] = j >= sp.lo && j < sp.hi ? 1.f : 0.f;
                }
            const typename TL::P ones = TL::weights(in);
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                const f32x4 up = TL::count_odd(vf, c, TL::kMinusInf, ones);
                const f32x4 down = TL::count_odd(vf, c, TL::kPlusInf, ones);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[c][e] += (up[e] > 0.f ? INFINITY : 0.f) + (down[e] > 0.f ? -INFINITY : 0.f);
                __builtin_amdgcn_sched_barrier(0);   // a rare path: few registers
            }
            TL::clear_odd(vf);
        }
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] = TL::pv(vf, c, p, acc[c]);
    };

    // Pages of the next 64 tiles from tile i0 on, `step` apart, one per lane
    // (of the table's entries past the length too, which block_src leaves out).
    constexpr int step = R == 1 ? kShares : 1;
    const int cap = a.map.max_pages << a.map.page_shift;
    int pg[kBlocks];
    auto load_pages = [&](int i0) {
        const int j = (tile0 + i0 + step * lane) * kTile;
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
            pg[blk] = j + 16 * blk < cap ? page_of(a.map, b, j + 16 * blk) : -1;
    };
    // the cache rows of block blk of tile i, whose pages lane `at` holds (none
    // past the length, on an absent page or past the last tile: such loads
    // give zeros)
    const size_t page_bytes = (size_t)TL::kRowBytes << a.map.page_shift;
    struct Src { size_t at; unsigned bytes; };
    auto block_src = [&](int i, int at, int blk) {
        const int page = __builtin_amdgcn_readlane(pg[blk], at);
        const int j = (tile0 + i) * kTile + 16 * blk;
        Src s;
        s.at = ((size_t)page * a.Hkv + h) * page_bytes + (size_t)slot_of(a.map, j) * TL::kRowBytes;
        const int valid = len - j < 16 ? len - j : 16;
        const bool some = page >= 0 && i < tiles && valid > 0;
        s.bytes = some ? (unsigned)(valid * TL::kRowBytes) : 0u;
        if (!some) s.at = 0;
        return s;
    };
    if constexpr (R == 1) {
        // D = 64: two tiles on their way, in two sets of registers.  D = 128:
        // one, as a second set's 64 registers would spill (64 contexts 125 ->
        // 136 us with it; D = 64 in fp32, 8 contexts: 35 -> 31 us).
        constexpr bool kTwo = D == 64;
        struct Ahead {
            typename TL::K kf;
            typename TL::V vf;
            Src src[kBlocks];
        } s0, s1;
        int at = 0;                             // tiles whose loads have been issued
        auto load_k = [&](Ahead &s) {
            if ((at & 63) == 0) load_pages(share + kShares * at);
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) {
                s.src[blk] = block_src(share + kShares * at, at & 63, blk);
                TL::load_k(s.kf, blk, make_rsrc(kc + s.src[blk].at, s.src[blk].bytes), lane);
            }
            ++at;
        };
        auto load_v = [&](Ahead &s) {
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk)
                TL::load_v(s.vf, blk, make_rsrc(vc + s.src[blk].at, s.src[blk].bytes), lane);
        };
        auto work = [&](int i, Ahead &s) {
            const int j0 = (tile0 + i) * kTile;
            f32x4 x[kBlocks];
            bool here[kBlocks], full = j0 >= all_lo && j0 + kTile <= all_hi;
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) {
                x[blk] = TL::logits(s.kf, blk, q);
                here[blk] = s.src[blk].bytes != 0;
                full &= here[blk];
            }
            load_k(s);
            absorb(j0, x, s.vf, full, here);
            load_v(s);
        };
        load_k(s0);
        load_v(s0);
        if constexpr (kTwo) {
            load_k(s1);
            load_v(s1);
        }
        for (int i = share; i < tiles; i += kShares) {
            work(i, s0);
            if constexpr (kTwo) {
                i += kShares;
                if (i >= tiles) break;
                work(i, s1);
            }
        }
    } else {
        constexpr int kChunks = TL::kRowBytes / 16, kUnits = kTileBytes / 16 / kThreads;
        static_assert(kUnits * kThreads * 16 == kTileBytes && 64 / kChunks <= 16,
                      "threads cover a tile, a wave's rows lie in one block");
        // a stage on its way: 16 bytes of K and of V per thread, unit and
        // share, and which blocks of this wave's own tile are there
        struct Stage {
            u32x4 kv[kShares][kUnits][2];
            bool here[kBlocks];
        };
        int paged = 0;                          // the tile that lane 0 of pg stands for
        load_pages(0);
        auto load = [&](int it, Stage &s) {
#pragma unroll
            for (int x = 0; x < kShares; ++x) {
                const int i = it * kShares + x;
                if (i >= paged + 64) {
                    paged = i;
                    load_pages(i);
                }
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const int unit = tid + kThreads * u, r = unit / kChunks;
                    const int blk = __builtin_amdgcn_readfirstlane(r >> 4);
                    const Src src = kBlocks == 1 || blk == 0 ? block_src(i, i - paged, 0)
                                                             : block_src(i, i - paged, kBlocks - 1);
                    const unsigned off = (r & 15) * TL::kRowBytes + unit % kChunks * 16;
                    s.kv[x][u][0] = __builtin_amdgcn_raw_buffer_load_b128(
                        make_rsrc(kc + src.at, src.bytes), off, 0, 0);
                    s.kv[x][u][1] = __builtin_amdgcn_raw_buffer_load_b128(
                        make_rsrc(vc + src.at, src.bytes), off, 0, 0);
                }
                if (x == share)
#pragma unroll
                    for (int blk = 0; blk < kBlocks; ++blk)
                        s.here[blk] = block_src(i, i - paged, blk).bytes != 0;
            }
        };
        auto store = [&](char *to, const Stage &s) {
#pragma unroll
            for (int x = 0; x < kShares; ++x)
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const int unit = tid + kThreads * u;
                    const int at = 2 * x * kTileBytes +
                                   chunk_at<TL::kRowBytes>(unit / kChunks, unit % kChunks);
                    *reinterpret_cast<u32x4 *>(to + at) = s.kv[x][u][0];
                    *reinterpret_cast<u32x4 *>(to + at + kTileBytes) = s.kv[x][u][1];
                }
        };
        typename TL::K kf;
        typename TL::V vf;
        auto work = [&](int it, const char *from, const bool (&here)[kBlocks]) {
            const int j0 = (tile0 + it * kShares + share) * kTile;
            const char *t = from + 2 * share * kTileBytes;
            f32x4 x[kBlocks];
            bool full = j0 >= all_lo && j0 + kTile <= all_hi;
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) {
                TL::lds_k(kf, blk, t, lane);
                TL::lds_v(vf, blk, t + kTileBytes, lane);
                full &= here[blk];
            }
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) x[blk] = TL::logits(kf, blk, q);
            absorb(j0, x, vf, full, here);
        };
        const int its = (tiles + kShares - 1) / kShares;
        Stage s0, s1;
        bool here0[kBlocks], here1[kBlocks];
        auto put = [&](char *to, const Stage &s, bool (&here)[kBlocks]) {
            store(to, s);
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) here[blk] = s.here[blk];
        };
        load(0, s0);
        load(1, s1);
        put(lds, s0, here0);
        load(2, s0);
        __syncthreads();
        for (int it = 0; it < its; it += 2) {
            work(it, lds, here0);
            put(lds + kStage, s1, here1);
            load(it + 3, s1);
            __syncthreads();
            if (it + 1 >= its) break;
            work(it + 1, lds + kStage, here1);
            put(lds, s0, here0);
            load(it + 4, s0);
            __syncthreads();
        }
        __syncthreads();                        // the stages make room for o
    }

    // join the waves of a row tile: every wave's o in units of their common
    // maximum, summed row by row
    l = swap_sum32(swap_sum16(l));
    if (lg == 0) {
        sm[w][r16] = m;
        sl[w][r16] = l;
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kShares; ++i) top = fmaxf(top, sm[rt + R * i][r16]);
    const float f = exp2_(m - finite_top(top));
    // acc[c][e] is channel dim(c, 4 lg + e); four at a time
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < PER; c += 4)
            *reinterpret_cast<f32x4 *>(&so[w][r16][TL::dim(c, 4 * lg + e)]) =
                f32x4{acc[c][e] * f, acc[c + 1][e] * f, acc[c + 2][e] * f, acc[c + 3][e] * f};
    __syncthreads();
    // 16 threads per row, four channels at a time
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int lr = tid >> 4, orow = row0 + 16 * i + lr;
        if (orow >= rows) break;
        float rtop = -INFINITY, rl = 0.f;
#pragma unroll
        for (int x = 0; x < kShares; ++x) rtop = fmaxf(rtop, sm[i + R * x][lr]);
#pragma unroll
        for (int x = 0; x < kShares; ++x)
            rl += sl[i + R * x][lr] * exp2_(sm[i + R * x][lr] - finite_top(rtop));
        const size_t part = ((size_t)slot * k.plan.units + h * k.plan.row_blocks + rb) * 16 * R +
                            16 * i + lr;
        const bool alone = sl_.count == 1;
        if ((!alone || k.logits) && (tid & 15) == 0) k.ml[part] = float2{rtop, rl};
        const float inv = 1.f / rl;
        const int t = orow / a.G, g = orow % a.G;
        T *o = static_cast<T *>(a.o) + (((size_t)b * a.n + t) * a.Hq + h * a.G + g) * D;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const int d = 64 * u + 4 * (tid & 15);
            f32x4 y = *reinterpret_cast<const f32x4 *>(&so[i][lr][d]);
#pragma unroll
            for (int x = 1; x < kShares; ++x)
                y += *reinterpret_cast<const f32x4 *>(&so[i + R * x][lr][d]);
            if (!alone) {
                *reinterpret_cast<f32x4 *>(k.po + part * D + d) = y;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = rl == 0.f ? 0.f : y[e] * inv;
                if constexpr (sizeof(T) == 2) *reinterpret_cast<bf16x4 *>(o + d) = cvt4(y);
                else                          *reinterpret_cast<f32x4 *>(o + d) = y;
            }
        }
    }
}

// (m, l) of one row over a sequence's slots, `stride` parts apart, by one
// wave: lanes take slots in turn.
__device__ inline float2 join_ml(const float2 *ml, size_t part, size_t stride, int count) {
    const int lane = threadIdx.x & 63;
    float top = -INFINITY, l = 0.f;
    for (int i = lane; i < count; i += 64) {
        const float2 x = ml[part + i * stride];
        const float mn = fmaxf(top, x.x), ms = finite_top(mn);
        l = l * exp2_(top - ms) + x.y * exp2_(x.x - ms);
        top = mn;
    }
    float all = top;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) all = fmaxf(all, __shfl_xor(all, m));
    all = finite_top(all);
    l *= exp2_(top - all);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) l += __shfl_xor(l, m);
    return float2{all, l};
}

// Joins the slots' parts, one workgroup per query row (the first `joins`
// workgroups): D / 4 threads across a row, the others across slots.  With
// scores, further workgroups each add the weights of 1,024 tokens of a
// (sequence, head): a thread sums 2^{x - m} / l over the rows, in their order,
// for four tokens.
template <typename T, int D, int R>
__global__ __launch_bounds__(kThreads) void join_kernel(KArgs k, long long joins,
                                                        long long score_blocks) {
    constexpr int kAcross = D / 4, kGroups = kThreads / kAcross;
    const AttnArgs &a = k.a;
    const int tid = threadIdx.x, rows = a.n * a.G;
    const size_t stride = (size_t)k.plan.units * 16 * R;
    if (blockIdx.x < joins) {
        __shared__ __align__(16) float so[kGroups][D];
        const long long q = blockIdx.x;
        const int hq = (int)(q % a.Hq), t = (int)(q / a.Hq % a.n), b = (int)(q / a.Hq / a.n);
        const int2 sc = k.sched[b];
        if (sc.y == 1) return;
        const int h = hq / a.G, row = t * a.G + hq % a.G;
        const int rb = row / (16 * R);
        const size_t part = (size_t)sc.x * stride + ((size_t)h * k.plan.row_blocks + rb) * 16 * R +
                            row % (16 * R);
        const float2 tot = join_ml(k.ml, part, stride, sc.y);
        const int d = 4 * (tid % kAcross), grp = tid / kAcross;
        f32x4 y{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int i = grp; i < sc.y; i += kGroups) {
            const float f = exp2_(k.ml[part + i * stride].x - tot.x);
            const f32x4 x = *reinterpret_cast<const f32x4 *>(k.po + (part + i * stride) * D + d);
            y += x * f;
        }
        *reinterpret_cast<f32x4 *>(&so[grp][d]) = y;
        __syncthreads();
        if (grp > 0) return;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) y += *reinterpret_cast<const f32x4 *>(&so[i][d]);
        const float inv = 1.f / tot.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = tot.y == 0.f ? 0.f : y[e] * inv;
        T *o = static_cast<T *>(a.o) + q * D + d;
        if constexpr (sizeof(T) == 2) *reinterpret_cast<bf16x4 *>(o) = cvt4(y);
        else                          *reinterpret_cast<f32x4 *>(o) = y;
        return;
    }
    constexpr int kRows = 64, kTokens = 4 * kThreads;
    __shared__ float2 st[kRows];
    const int w = tid >> 6;
    const long long per = (k.cap32 + kTokens - 1) / kTokens;
    const long long all = (long long)a.B * a.Hkv * per;
    for (long long blk = blockIdx.x - joins; blk < all; blk += score_blocks) {
        const int bh = (int)(blk / per), b = bh / a.Hkv, h = bh % a.Hkv;
        const int len = cached_len(a.seq_lens, b, a.map);
        const Span seq = seq_span(len, a.n, a.window);
        const int base = (int)(blk % per) * kTokens;
        if (base >= len || base + kTokens <= seq.lo) continue;    // the same for all threads
        const int2 sc = k.sched[b];
        const int j = base + 4 * tid;
        f32x4 sum{0.f, 0.f, 0.f, 0.f};
        for (int r0 = 0; r0 < rows; r0 += kRows) {
            const int nr = rows - r0 < kRows ? rows - r0 : kRows;
            __syncthreads();
            for (int r = w; r < nr; r += kWaves) {
                const int row = r0 + r;
                const size_t part = (size_t)sc.x * stride +
                                    ((size_t)h * k.plan.row_blocks + row / (16 * R)) * 16 * R +
                                    row % (16 * R);
                const float2 x = join_ml(k.ml, part, stride, sc.y);
                if ((tid & 63) == 0) st[r] = float2{x.x, x.y == 0.f ? 0.f : 1.f / x.y};
            }
            __syncthreads();
            if (j < len) {
                const float *x = k.logits + (((size_t)b * a.Hkv + h) * rows + r0) * k.cap32 + j;
#pragma unroll 4
                for (int r = 0; r < nr; ++r) {
                    const Span sp = token_span(len, a.n, a.window, (r0 + r) / a.G);
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(x + r * k.cap32);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e >= sp.lo && j + e < sp.hi) sum[e] += exp2_(v[e] - st[r].x) * st[r].y;
                }
            }
        }
        if (j < len) {
            const int page = page_of(a.map, b, j);
            const int lo = token_span(len, a.n, a.window, 0).lo;
            if (page >= 0) {
                float *s = a.scores + cache_row(a.map, a.Hkv, page, h, slot_of(a.map, j));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e >= lo && j + e < len) s[e] += sum[e];
            }
        }
    }
}

template <typename T, int D, int R>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    const long long cap = (long long)a.map.max_pages << a.map.page_shift;
    const WsMap w = ws_map(a.B, a.n, a.G, a.Hkv, D, R, cap, a.scores != nullptr);
    char *ws = static_cast<char *>(a.ws);
    KArgs k{};
    k.a = a;
    k.plan = make_plan(a.B, a.n, a.G, a.Hkv, R, cap);
    k.sched = reinterpret_cast<int2 *>(ws + w.sched);
    k.ml = reinterpret_cast<float2 *>(ws + w.ml);
    k.po = reinterpret_cast<float *>(ws + w.o);
    k.logits = a.scores ? reinterpret_cast<float *>(ws + w.logits) : nullptr;
    k.cap32 = (cap + 31) / 32 * 32;
    k.parts = k.plan.max_slots > a.B;
    const long long pairs = ((long long)k.plan.max_slots * a.Hkv + 7) / 8 * 8;
    attn_kernel<T, D, R><<<(unsigned)(pairs * k.plan.row_blocks), kThreads, 0, s>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long joins = k.parts ? (long long)a.B * a.n * a.Hq : 0;
    long long score_blocks = a.scores ? (long long)a.B * a.Hkv * ((k.cap32 + 1023) / 1024) : 0;
    if (score_blocks > (1 << 20)) score_blocks = 1 << 20;
    if (joins + score_blocks == 0) return hipSuccess;
    join_kernel<T, D, R><<<(unsigned)(joins + score_blocks), kThreads, 0, s>>>(k, joins, score_blocks);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_r(const AttnArgs &a, hipStream_t s) {
    switch (row_tiles((long long)a.n * a.G)) {
    case 1:  return launch<T, D, 1>(a, s);
    case 2:  return launch<T, D, 2>(a, s);
    default: return launch<T, D, 4>(a, s);
    }
}

}  // namespace

size_t attention_workspace(int B, int n, int Hq, int Hkv, int D, long long capacity,
                           bool with_scores) {
    const int G = Hq / Hkv;
    return ws_map(B, n, G, Hkv, D, row_tiles((long long)n * G), capacity, with_scores).total;
}

hipError_t launch_attention_decode(bool bf16_io, int D, const AttnArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? launch_r<bf16, 128>(a, s) : launch_r<bf16, 64>(a, s);
    return D == 128 ? launch_r<float, 128>(a, s) : launch_r<float, 64>(a, s);
}

}  // namespace gdr

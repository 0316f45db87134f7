// attention.hip -- attention of new tokens over the paged key-value cache,
// for gfx950.
//
// Row (b, t, h) of the queries stands at position p = len_b - n + t and
// attends to the cached tokens j <= p (and j > p - window):
//     s_j = scale q.k_j,   w_j = e^{s_j} / sum e^{s_i},   o = sum w_j v_j.
//
// One pass over K and V with a running maximum m and sum l: with c = |scale|
// log2 e (a negative scale's sign goes into q) and y = q.k, for a tile of
// tokens m' = max(m, max y), l = l 2^{c (m - m')} + sum 2^{c (y - m')}, o
// likewise.  Parts of a sequence join by the same rule.  (The difference is
// taken before the product: near the maximum, where the weights are, it is
// exact.)
//
// The G = Hq / Hkv query heads of a key-value head and the n new tokens make
// n G rows that read the same K and V: a workgroup has up to 32 of them (16 in
// fp32), so that a token is read from HBM once for all of them, as MFMA
// operands.  Bytes bound the kernel: 2 D elements a token against 4 D flops
// per row and token is at most 32 flops a byte, where the card turns at
// about 250.  64 contexts of 512 to 8,192 tokens, 8 heads of 128 in bf16 (681
// MB): 118 us, 5.8 TB/s, where a plain read of that size reaches 6.2 to 6.5 and
// a copy 5.0; the same with K and V only loaded: 112 us.
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
// chunks of about C tokens, the same C for all, so that a long sequence among
// short ones is spread over as many workgroups as its length asks for; C
// follows from the lengths on the device.  Chunks are numbered over the
// sequences ("slots"); a sequence without tokens has one, which writes its
// zeros.
//   The card holds kResident workgroups at once, and workgroups of a like
// size end together: with sum ceil(len / C) <= total / C + B slots, C is taken
// such that they fill the card once, or twice or four times where B
// sequences' last chunks would leave over a quarter of it idle (130,001
// tokens: 57 us with C for 1,024 workgroups, 52 us so).  With more sequences
// than that, C is for 1,024.
//   Which slot is whose each workgroup finds for itself from the lengths, or,
// with more than kScan sequences, a launch before finds for all (4,096
// sequences of up to 1,000 tokens: 461 us and 378 us).  Past kMaxShared
// sequences each is one slot.
constexpr int kResident = 512;
constexpr int kScan = 256;
constexpr int kMaxShared = 1 << 16;
constexpr int kMinChunk = 512;
struct Plan {
    int units;            // workgroups of one slot: key-value heads x row blocks
    int row_blocks;       // blocks of RW rows
    int want_slots;       // total / C
    int max_slots;        // bound on the slots there can be: sum ceil(len / C) <= want + B
};
Plan make_plan(int B, int n, int G, int Hkv, int rw, long long capacity) {
    Plan p;
    p.row_blocks = (n * G + rw - 1) / rw;
    p.units = Hkv * p.row_blocks;
    p.want_slots = 2 * kResident / p.units;
    for (int k = 4; k >= 1; k >>= 1)
        if (4LL * B * p.units <= k * kResident) p.want_slots = k * kResident / p.units - B;
    if (p.want_slots < 1) p.want_slots = 1;
    const long long by_len = (capacity + kMinChunk - 1) / kMinChunk * B;
    const long long bound = (long long)p.want_slots + B;
    p.max_slots = (int)(by_len < bound ? (by_len < B ? B : by_len) : bound);
    if (B > kMaxShared) p.max_slots = B;
    return p;
}
// Rows of a workgroup's block (RW), those of one MFMA tile.  More rows are
// several blocks, which read K and V from L2 after the first.  In fp32 a block
// of 32 would need twice the registers there are.
//   Over 32 rows with much to read, 64: two tiles of rows share the tokens
// through LDS (16 new tokens, 4 heads of 4 rows each, from cold caches: 16
// contexts of 2,000 tokens 31 us against 46 in blocks of 32, of 1,500 30
// against 37, 2 of 16,000 29 against 42).  With little to read the two blocks
// side by side are done sooner (16 contexts of 1,000: 26 us against 29; one of
// 300: 12 against 16).  The lengths are on the device, so what the table and
// the window let a sequence attend to decides, and short contexts under a wide
// table lose by it (the one of 300 under a table of 131,072 tokens, a call
// with its second launch: 18 us, 10 under a table of its length; 16 of 300 to
// 1,000 with 8 heads: 29 either way).
constexpr long long kShareBytes = 40LL << 20;
int block_rows(bool bf16_io, long long rows, int B, int n, int Hkv, int D, long long capacity,
               int window) {
    if (!bf16_io || rows <= 16) return 16;
    const long long seen = window > 0 && window < capacity - n ? window + n : capacity;
    return rows > 32 && seen * B * Hkv * D * 4 >= kShareBytes ? 64 : 32;
}

// Workspace: {first slot, slots} of every sequence; with more than kScan of
// them, every slot's {sequence, its first slot, its slots, tokens of one};
// (m, l) of every slot, unit and row; o of the same, unnormalised; with
// scores, the products q.k of every row and token [B, Hkv, nG, cap].  Of a
// table without pages, nothing: there is one launch, which writes none of it.
struct WsMap {
    size_t sched, slots, ml, o, logits, total;
};
WsMap ws_map(int B, int n, int G, int Hkv, int D, int rw, long long capacity, bool with_scores) {
    auto r256 = [](size_t x) { return (x + 255) / 256 * 256; };
    WsMap w{};
    if (capacity == 0) return w;
    const Plan p = make_plan(B, n, G, Hkv, rw, capacity);
    const size_t rows = (size_t)p.max_slots * p.units * rw;
    const bool parts = p.max_slots > B;
    w.sched = 0;
    w.slots = r256((size_t)B * 2 * sizeof(int));
    w.ml = w.slots + (parts && B > kScan ? r256((size_t)p.max_slots * sizeof(int4)) : 0);
    w.o = w.ml + (parts || with_scores ? r256(rows * 2 * sizeof(float)) : 0);
    w.logits = w.o + (parts ? r256(rows * D * sizeof(float)) : 0);
    w.total = w.logits + (with_scores ? (size_t)B * Hkv * n * G * ((capacity + 31) / 32 * 32) *
                                            sizeof(float) : 0);
    return w;
}

struct KArgs {
    AttnArgs a;
    Plan plan;
    int2 *sched;          // nullptr: a table without pages
    int4 *slots;          // nullptr: found by each workgroup
    float2 *ml;
    float *po;
    float *logits;        // nullptr: no scores
    long long cap32;      // tokens of a logits row
    float c;              // |scale| log2 e, above 0
    bool negative;        // scale < 0
    bool parts;           // a sequence may have several slots
};

// Sum over the workgroup's threads before this one and over all; lds holds a
// value per wave.
template <int WAVES, typename N>
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
    for (int i = 0; i < WAVES; ++i) {
        const N v = lds[i];
        before += i < w ? v : 0;
        total += v;
    }
    __syncthreads();
    return before + incl - x;
}

// A value that is the same in all lanes, for a scalar register.
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

struct Slot { int b, first, count, chunk; };      // sequence, its first slot, its slots, tokens of one

// Shares the sequences' slots out over a workgroup of 64 WAVES threads, thread
// t looking after sequences t per .. t per + per - 1: begin() gives the
// thread's first slot and all slots, next() goes through its sequences.
template <int WAVES>
struct Sharing {
    const KArgs &k;
    int per, b, end, at, chunk;
    __device__ Sharing(const KArgs &k) : k(k) {
        per = (k.a.B + 64 * WAVES - 1) / (64 * WAVES);
        b = threadIdx.x * per;
        end = b + per < k.a.B ? b + per : k.a.B;
    }
    __device__ inline int tokens(int i) const {
        const AttnArgs &a = k.a;
        const Span sp = seq_span(cached_len(a.seq_lens, i, a.map), a.n, a.window);
        return sp.hi - sp.lo;
    }
    __device__ inline int slots_of(int tok) const {
        const int n = (tok + chunk - 1) / chunk;
        return n > 1 ? n : 1;
    }
    // returns all slots
    __device__ inline int begin(int &mine) {
        __shared__ long long lds64[WAVES];
        __shared__ int lds32[WAVES];
        long long sum = 0, total;
#pragma unroll 4
        for (int i = b; i < end; ++i) sum += tokens(i);
        group_scan<WAVES, long long>(sum, total, lds64);
        long long c = (total + k.plan.want_slots - 1) / k.plan.want_slots;
        c = c < kMinChunk ? kMinChunk : (c > (1 << 30) ? 1 << 30 : c);
        chunk = (int)((c + 127) / 128 * 128);
        mine = 0;
        int all;
#pragma unroll 4
        for (int i = b; i < end; ++i) mine += slots_of(tokens(i));
        at = group_scan<WAVES, int>(mine, all, lds32);
        return all;
    }
    // the slots of sequence b: alike, in multiples of 128 tokens
    __device__ inline Slot next() {
        const int tok = tokens(b), n = slots_of(tok);
        const Slot s{b, at, n, ((tok + n - 1) / n + 127) & ~127};
        ++b;
        at += n;
        return s;
    }
};

// Every slot's owner, by one workgroup for all.
__global__ __launch_bounds__(1024) void slots_kernel(KArgs k) {
    Sharing<16> sh(k);
    int mine;
    const int all = sh.begin(mine);
    while (sh.b < sh.end) {
        const Slot s = sh.next();
        for (int i = 0; i < s.count; ++i) k.slots[s.first + i] = int4{s.b, s.first, s.count, s.chunk};
    }
    for (int i = all + threadIdx.x; i < k.plan.max_slots; i += 1024) k.slots[i] = int4{-1, 0, 0, 0};
}

// The sequence that slot s belongs to (b = -1: past the last slot).
__device__ inline Slot find_slot(const KArgs &k, int s) {
    // no sequence has a second slot: slot and sequence are one
    if (!k.parts) return Slot{s < k.a.B ? s : -1, s, 1, 1 << 30};
    if (k.slots) {
        if (s >= k.plan.max_slots) return Slot{-1, 0, 0, 0};
        const int4 x = k.slots[s];
        return Slot{uniform(x.x), uniform(x.y), uniform(x.z), uniform(x.w)};
    }
    __shared__ Slot found;
    if (threadIdx.x == 0) found.b = -1;
    Sharing<kWaves> sh(k);
    int mine;
    sh.begin(mine);
    if (s >= sh.at && s < sh.at + mine) {
        Slot x;
        do x = sh.next(); while (s >= sh.at);
        found = x;
    }
    __syncthreads();
    return Slot{uniform(found.b), uniform(found.first), uniform(found.count), uniform(found.chunk)};
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

// K and V that one workgroup reads once pass through the caches without
// staying there (64 contexts of 4,096 tokens: 169 us, 195 without the hint);
// what several row blocks read is kept.  Which pages sequences share only the
// device knows: of shared ones the caches then keep less (half of each context
// shared by all 64: 137 us, 121 without the hint).
template <bool STREAM>
__device__ inline u32x4 load16(rsrc_t r, unsigned off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, STREAM ? 2 : 0);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// A block of 16 tokens of one head in a cache: its first byte, and how many
// bytes of it may be read (0: none of its tokens are there).
struct Src { size_t at; unsigned bytes; };

// A tile of tokens as MFMA operands, per dtype and rows of a block.  With RW
// rows, lane = RW g + r is row r:
//   S^T = K Q^T: the lane supplies key r (A) and query row r (B), and gets
//     logits of query row r: value i is that of the tile's token key(i, g);
//   O^T = V^T P^T: P^T's operand is those logits' weights as they lie (the
//     sum over k runs over the keys in whatever order both operands use),
//     and V^T's is read from the rows of V that hold the same keys, PER = D / RW
//     channels per lane, so that V needs no transposition through LDS:
//     acc[c][i] is channel dim(c, m(i, g)) of query row r.
template <typename T, int D, int RW> struct Tile;

// two keys' values of one channel pair -> channel c of both
__device__ inline unsigned pick2(unsigned k0, unsigned k1, int c) {
    return __builtin_amdgcn_perm(k1, k0, c & 1 ? 0x07060302u : 0x05040100u);
}
// bits 15 and 31: whether the word's bf16 values are infinities or NaN (an
// exponent of all ones carries)
__device__ inline unsigned odd2(unsigned x) { return (x & 0x7F807F80u) + 0x00800080u; }
__device__ inline unsigned clear2(unsigned x) {
    return ((x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) |
           ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u);
}
// 1 where a value is an infinity or NaN other than `but`
__device__ inline unsigned mark2(unsigned x, unsigned but) {
    const unsigned lo = x & 0xFFFFu, hi = x >> 16;
    return ((lo & 0x7F80u) == 0x7F80u && lo != but ? 0x3F80u : 0u) |
           ((hi & 0x7F80u) == 0x7F80u && hi != but ? 0x3F800000u : 0u);
}

template <int D, int RW> struct Tile<bf16, D, RW> {
    static constexpr int kBlocks = 2, kTile = 32;  // blocks of 16 tokens
    static constexpr int kGroups = 64 / RW;        // lanes of a row
    static constexpr int kVals = kTile / kGroups;  // logits of a lane
    static constexpr int PER = D / RW;             // channels of a lane's V rows, blocks of acc
    static constexpr int kRowBytes = D * 2;
    // a row in LDS: 16 bytes more, so that the rows of a K operand start in
    // different banks
    static constexpr int kPitch = kRowBytes + 16;
    static constexpr int kSteps = D / (8 * kGroups);     // MFMAs of a block of keys
    static constexpr int kKeyBlocks = kTile / RW;        // S^T tiles: 2 (RW = 16) or 1
    typedef std::conditional_t<RW == 16, f32x4, f32x16> Acc;
    static constexpr int kAcc = sizeof(Acc) / 4;
    struct Q { bf16x8 f[kSteps]; };
    struct K { bf16x8 f[kKeyBlocks][kSteps]; };
    struct V { unsigned w[kVals][PER / 2]; };      // row of V: key(i, g)
    // RW = 16: blocks of 16 keys, 4 g + e each; RW = 32: 8 (e / 4) + 4 g + e % 4
    __device__ static inline int key(int i, int g) {
        return RW == 16 ? 16 * (i >> 2) + 4 * g + (i & 3) : 8 * (i >> 2) + 4 * g + (i & 3);
    }
    __device__ static inline int dim(int c, int i, int g) {
        return PER * (RW == 16 ? 4 * g + i : 8 * (i >> 2) + 4 * g + (i & 3)) + c;
    }
    static constexpr int block(int i) { return RW == 16 ? i >> 2 : i >> 3; }   // key's block of 16
    __device__ static inline Acc mfma(bf16x8 a, bf16x8 b, Acc c) {
        if constexpr (RW == 16) return mfma32(a, b, c);
        else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    __device__ static inline void load_q(Q &q, rsrc_t r, unsigned off, int lane) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) q.f[i] = bload16(r, off + 16 * kGroups * i + 16 * (lane / RW));
    }
    __device__ static inline void negate(Q &q) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            q.f[i] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, q.f[i]) ^ 0x80008000u);
    }
    // kc + src[b].at: the rows of block b of 16 tokens
    template <bool STREAM>
    __device__ static inline void load_k(K &k, const char *kc, const Src (&src)[2], bool one_page,
                                         int lane) {
        const int g = lane / RW, r = lane % RW;
        if constexpr (RW == 16) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const rsrc_t rs = make_rsrc(kc + src[b].at, src[b].bytes);
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
                    k.f[b][i] = __builtin_bit_cast(
                        bf16x8, load16<STREAM>(rs, r * kRowBytes + 16 * kGroups * i + 16 * g));
            }
        } else if (one_page) {
            // both blocks, one after the other
            const rsrc_t whole = make_rsrc(kc + src[0].at, src[0].bytes + src[1].bytes);
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                k.f[0][i] = __builtin_bit_cast(
                    bf16x8, load16<STREAM>(whole, r * kRowBytes + 16 * kGroups * i + 16 * g));
        } else if (src[0].bytes + src[1].bytes) {
            // pages of 16: an address per lane.  Rows of an absent block are
            // read from the other one, and rows past the length as they lie
            // in their page: their logits are masked.
            const bool second = r < 16 ? src[0].bytes == 0 : src[1].bytes != 0;
            const u32x4 *p = reinterpret_cast<const u32x4 *>(
                kc + (second ? src[1].at : src[0].at) + (r & 15) * kRowBytes + 16 * g);
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                k.f[0][i] = __builtin_bit_cast(bf16x8, STREAM ? __builtin_nontemporal_load(p + kGroups * i)
                                                              : p[kGroups * i]);
        }
    }
    template <bool STREAM>
    __device__ static inline void load_v(V &v, const rsrc_t (&rsrc)[2], int lane) {
        const int g = lane / RW, r = lane % RW;
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const unsigned off = (key(i, g) & 15) * kRowBytes + r * PER * 2;
            if constexpr (PER == 8) {
                const u32x4 x = load16<STREAM>(rsrc[block(i)], off);
#pragma unroll
                for (int j = 0; j < 4; ++j) v.w[i][j] = x[j];
            } else if constexpr (PER == 4) {
                const auto x = __builtin_amdgcn_raw_buffer_load_b64(rsrc[block(i)], off, 0, STREAM ? 2 : 0);
                v.w[i][0] = x[0];
                v.w[i][1] = x[1];
            } else {
                v.w[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc[block(i)], off, 0, STREAM ? 2 : 0);
            }
        }
    }
    // the same from a tile that lies in LDS (RW = 32)
    __device__ static inline void lds_k(K &k, const char *t, int lane) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            k.f[0][i] = *reinterpret_cast<const bf16x8 *>(
                t + lane % RW * kPitch + 16 * (kGroups * i + lane / RW));
    }
    __device__ static inline void lds_v(V &v, const char *t, int lane) {
        const int g = lane / RW, at = lane % RW * PER * 2;
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const char *p = t + key(i, g) * kPitch + at;
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) v.w[i][j] = reinterpret_cast<const unsigned *>(p)[j];
        }
    }
    __device__ static inline void logits(float (&x)[kVals], const K &k, const Q &q) {
#pragma unroll
        for (int b = 0; b < kKeyBlocks; ++b) {
            Acc s;
#pragma unroll
            for (int e = 0; e < kAcc; ++e) s[e] = 0.f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s = mfma(k.f[b][i], q.f[i], s);
#pragma unroll
            for (int e = 0; e < kAcc; ++e) x[kAcc * b + e] = s[e];
        }
    }
    // Weights as the sum of two bf16 numbers, the product's operands: hi, cut
    // to bf16, and lo, the rest rounded to it, together off by at most 2^-15 of
    // a weight (one bf16 number: 2^-8).  The rest gains 2^-23 of the weight, so
    // that lo is above 0 where the weight is (2^-103 or more, which leaves it a
    // normal number) and an infinity of V that a row attends to meets no 0 of a
    // weight that one number holds.
    //   The second product costs nothing where bytes bound the call (64 contexts
    // 120 us either way), 7 % in blocks of 64 rows (55 -> 59 us), and brings o
    // from 1.08 to 1.00 times the error of fp32 weights against 64 bits.
    struct P { bf16x8 hi[kVals / 8], lo[kVals / 8]; };
    __device__ static inline P weights(const float (&x)[kVals]) {
        P p;
#pragma unroll
        for (int h = 0; h < kVals / 8; ++h) {
            u32x4 hi;
            float lo[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float a = x[8 * h + 2 * u], b = x[8 * h + 2 * u + 1];
                const unsigned ab = __builtin_bit_cast(unsigned, a), bb = __builtin_bit_cast(unsigned, b);
                hi[u] = __builtin_amdgcn_perm(bb, ab, 0x07060302u);
                lo[2 * u] = fmaf(a, 1.f + 0x1p-23f, -__builtin_bit_cast(float, ab & 0xFFFF0000u));
                lo[2 * u + 1] = fmaf(b, 1.f + 0x1p-23f, -__builtin_bit_cast(float, bb & 0xFFFF0000u));
            }
            p.hi[h] = __builtin_bit_cast(bf16x8, hi);
            p.lo[h] = cvt8(lo);
        }
        return p;
    }
    // 0 and 1
    struct Ones { bf16x8 f[kVals / 8]; };
    __device__ static inline Ones ones(const float (&x)[kVals]) {
        Ones p;
#pragma unroll
        for (int h = 0; h < kVals / 8; ++h) p.f[h] = cvt8(x + 8 * h);
        return p;
    }
    __device__ static inline u32x4 v_frag(const V &v, int c, int h) {
        u32x4 x;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = pick2(v.w[8 * h + 2 * u][c >> 1], v.w[8 * h + 2 * u + 1][c >> 1], c);
        return x;
    }
    __device__ static inline Acc pv(const V &v, int c, const P &p, Acc acc) {
#pragma unroll
        for (int h = 0; h < kVals / 8; ++h) {
            const bf16x8 x = __builtin_bit_cast(bf16x8, v_frag(v, c, h));
            acc = mfma(x, p.hi[h], acc);
            acc = mfma(x, p.lo[h], acc);
        }
        return acc;
    }
    // an infinity or NaN among this lane's values
    __device__ static inline bool odd(const V &v) {
        unsigned y = 0;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) y |= odd2(v.w[i][j]);
        return (y & 0x80008000u) != 0;
    }
    // how many infinities and NaN other than `but` (an infinity's bits) each
    // row meets where ones is 1
    __device__ static inline Acc count_odd(const V &v, int c, unsigned but, const Ones &ones) {
        Acc s;
#pragma unroll
        for (int e = 0; e < kAcc; ++e) s[e] = 0.f;
#pragma unroll
        for (int h = 0; h < kVals / 8; ++h) {
            u32x4 x = v_frag(v, c, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = mark2(x[i], but);
            s = mfma(__builtin_bit_cast(bf16x8, x), ones.f[h], s);
        }
        return s;
    }
    static constexpr unsigned kPlusInf = 0x7F80u, kMinusInf = 0xFF80u;
    __device__ static inline void clear_odd(V &v) {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) v.w[i][j] = clear2(v.w[i][j]);
    }
};

template <int D> struct Tile<float, D, 16> {
    static constexpr int kBlocks = 1, kTile = 16;
    static constexpr int kGroups = 4, kVals = 4, PER = D / 16, kRowBytes = D * 4;
    typedef f32x4 Acc;
    static constexpr int kAcc = 4;
    struct Q { f32x4 f[D / 16]; };
    struct K { f32x4 f[D / 16]; };
    struct V { f32x4 f[4][PER / 4]; };
    __device__ static inline int key(int i, int g) { return 4 * g + i; }
    static constexpr int block(int) { return 0; }
    // channels 64 (c / 4) + 4 m + c % 4: a load covers 256 bytes of a row
    __device__ static inline int dim(int c, int i, int g) {
        return 64 * (c >> 2) + 4 * (4 * g + i) + (c & 3);
    }
    // a value parameter: the bit cast of a vector's element in place takes
    // the vector's first element
    __device__ static inline unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }
    __device__ static inline f32x4 mfma(float a, float b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
    }
    __device__ static inline void load_q(Q &q, rsrc_t r, unsigned off, int lane) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) q.f[i] = bload16f(r, off + 64 * i + 16 * (lane >> 4));
    }
    __device__ static inline void negate(Q &q) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) q.f[i] = -q.f[i];
    }
    template <bool STREAM>
    __device__ static inline void load_k(K &k, const char *kc, const Src (&src)[1], bool, int lane) {
        const rsrc_t rs = make_rsrc(kc + src[0].at, src[0].bytes);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            k.f[i] = __builtin_bit_cast(
                f32x4, load16<STREAM>(rs, (lane & 15) * kRowBytes + 64 * i + 16 * (lane >> 4)));
    }
    template <bool STREAM>
    __device__ static inline void load_v(V &v, const rsrc_t (&rsrc)[1], int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                v.f[e][i] = __builtin_bit_cast(
                    f32x4, load16<STREAM>(rsrc[0], (4 * (lane >> 4) + e) * kRowBytes + 256 * i +
                                                       16 * (lane & 15)));
    }
    // four sums of D / 4 products, then their sum: a quarter of the roundings
    // on one sum's way (o's error against 64 bits 1.1e-6 -> 4.2e-7 relative for
    // 128 channels, 7.4e-7 -> 3.9e-7 for 64), in the same time
    __device__ static inline void logits(float (&x)[4], const K &k, const Q &q) {
        f32x4 s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = mfma(k.f[i][e], q.f[i][e], s[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (s[0][e] + s[1][e]) + (s[2][e] + s[3][e]);
    }
    struct P { float f[4]; };
    typedef P Ones;
    __device__ static inline P weights(const float (&x)[4]) { return P{{x[0], x[1], x[2], x[3]}}; }
    __device__ static inline Ones ones(const float (&x)[4]) { return weights(x); }
    __device__ static inline f32x4 pv(const V &v, int c, const P &p, f32x4 acc) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma(v.f[e][c >> 2][c & 3], p.f[e], acc);
        return acc;
    }
    __device__ static inline bool odd(const V &v) {
        bool y = false;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < PER; ++c)
                y |= (bits(v.f[e][c >> 2][c & 3]) & 0x7F800000u) == 0x7F800000u;
        return y;
    }
    __device__ static inline f32x4 count_odd(const V &v, int c, unsigned but, const Ones &ones) {
        f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned u = bits(v.f[e][c >> 2][c & 3]);
            s = mfma((u & 0x7F800000u) == 0x7F800000u && u != but ? 1.f : 0.f, ones.f[e], s);
        }
        return s;
    }
    static constexpr unsigned kPlusInf = 0x7F800000u, kMinusInf = 0xFF800000u;
    __device__ static inline void clear_odd(V &v) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                const unsigned u = bits(v.f[e][c >> 2][c & 3]);
                v.f[e][c >> 2][c & 3] = (u & 0x7F800000u) == 0x7F800000u ? 0.f : v.f[e][c >> 2][c & 3];
            }
    }
};

// Workgroup = (slot, key-value head, block of RW RT rows).  Its four waves are
// RT tiles of rows times 4 / RT shares, which take the slot's tiles of tokens
// in turn, each wave with m, l and o of its own, joined through LDS at the end.
//   RT = 1: K and V go from HBM straight into the registers that MFMA reads:
// the next tile to come is requested into a tile's registers as they fall
// free, K after its logits are formed, V after its product.  The 180 registers of
// a thread (RW = 16, D = 128) let two workgroups share a CU, 64 KiB on their way
// in each; three, by spilling, measured 141 us where two take 120 (64 contexts).
//   RT = 2: two waves read each tile, which all threads bring into LDS
// together, a stage (a tile per share) at a time: one stage is worked on while
// the next comes into registers, to be written beside it.  (16 contexts of
// 1,000 to 6,000, 64 rows a head: 59 us; with one bf16 number a weight 55, and
// 74 with RT = 1.  Rows in LDS are
// padded rather than exchanged: with a 16-byte chunk's place depending on its
// row by an exclusive or, the addresses alone took so many registers that 34
// others were spilled, 62 us.)
template <typename T, int D, int RW, int RT, bool STREAM>
__global__ __launch_bounds__(kThreads, 2) void attn_kernel(KArgs k) {
    using TL = Tile<T, D, RW>;
    constexpr int PER = TL::PER, kBlocks = TL::kBlocks, kTile = TL::kTile, kVals = TL::kVals;
    constexpr int kPad = D + 4, kShares = kWaves / RT, kRows = RW * RT;
    constexpr int kPitch = TL::kRowBytes + 16, kTileBytes = kTile * kPitch;
    constexpr int kStage = kShares * 2 * kTileBytes;
    constexpr int kOBytes = kWaves * RW * kPad * (int)sizeof(float);
    __shared__ float sm[kWaves][RW], sl[kWaves][RW];
    // the two stages, and at the end every wave's o
    __shared__ __align__(16) char lds[RT > 1 && 2 * kStage > kOBytes ? 2 * kStage : kOBytes];
    float(*so)[RW][kPad] = reinterpret_cast<float(*)[RW][kPad]>(lds);
    const AttnArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane % RW, g = lane / RW;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), rt = w % RT, share = w / RT;
    // the row blocks of one (slot, head) follow each other on one XCD, which
    // holds their K and V in its L2 (workgroups go to the eight XCDs in turn)
    const int wg = blockIdx.x;
    const int rb = wg / 8 % k.plan.row_blocks;
    const int unit = wg / 8 / k.plan.row_blocks * 8 + wg % 8;
    const int slot = unit / a.Hkv, h = unit % a.Hkv;
    const Slot sl_ = find_slot(k, slot);
    const int b = sl_.b;
    if (b < 0) return;
    const int len = uniform(cached_len(a.seq_lens, b, a.map));
    const Span seq = seq_span(len, a.n, a.window);
    if (k.sched && h == 0 && rb == 0 && slot == sl_.first && tid == 0)
        k.sched[b] = int2{sl_.first, sl_.count};

    // this lane's query row and what it attends to
    const int rows = a.n * a.G, row0 = rb * kRows, row = row0 + RW * rt + r;
    Span sp{0, 0};
    typename TL::Q q;
    {
        const size_t qb = (size_t)b * a.n * a.Hq * D;
        const rsrc_t rq = make_rsrc(static_cast<const T *>(a.q) + qb, 0xFFFFFFFFu);
        const int t = row < rows ? row / a.G : 0, hg = row < rows ? row % a.G : 0;
        if (row < rows) sp = token_span(len, a.n, a.window, t);
        TL::load_q(q, rq, (unsigned)(t * a.Hq + h * a.G + hg) * (D * (unsigned)sizeof(T)), lane);
        if (k.negative) TL::negate(q);
    }
    // the block's tokens: what its rows attend to, within the slot
    const Span first = token_span(len, a.n, a.window, row0 / a.G);
    const Span last = token_span(len, a.n, a.window,
                                 ((row0 + kRows < rows ? row0 + kRows : rows) - 1) / a.G);
    const int c_lo = seq.lo + (slot - sl_.first) * sl_.chunk;
    const int c_hi = c_lo + sl_.chunk < len ? c_lo + sl_.chunk : len;
    const int k_lo = first.lo > c_lo ? first.lo : c_lo, k_hi = last.hi < c_hi ? last.hi : c_hi;
    // every row attends to the tokens of [all_lo, all_hi)
    const int all_lo = last.lo, all_hi = first.hi;
    const int tile0 = k_lo / kTile;
    const int tiles = k_hi > k_lo ? (k_hi + kTile - 1) / kTile - tile0 : 0;

    const char *kc = static_cast<const char *>(a.k_cache), *vc = static_cast<const char *>(a.v_cache);
    float m = -INFINITY, l = 0.f;
    typename TL::Acc acc[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c)
#pragma unroll
        for (int e = 0; e < TL::kAcc; ++e) acc[c][e] = 0.f;

    // the largest of a value over a row's lanes, and the sum
    auto row_max = [](float x) { return swap_max32(RW == 16 ? swap_max16(x) : x); };
    auto row_sum = [](float x) { return swap_sum32(RW == 16 ? swap_sum16(x) : x); };

    // One tile's products q.k and values into m, l and o.  full:
    // every row attends to all of it; here: which of its blocks are there.
    // (Past the length and on absent pages V is zeros.)
    auto absorb = [&](int j0, float (&x)[kVals], typename TL::V &vf, bool full,
                      const bool (&here)[kBlocks]) {
        float top = -INFINITY;
        if (k.logits && row < rows) {
#pragma unroll
            for (int i = 0; i < kVals; i += 4)
                if (here[TL::block(i)])
                    *reinterpret_cast<f32x4 *>(k.logits +
                                               (((size_t)b * a.Hkv + h) * rows + row) * k.cap32 + j0 +
                                               TL::key(i, g)) = f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
        }
        if (!full) {
#pragma unroll
            for (int i = 0; i < kVals; ++i) {
                const int j = j0 + TL::key(i, g);
                x[i] = here[TL::block(i)] && j >= sp.lo && j < sp.hi ? x[i] : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) top = fmaxf(top, x[i]);
        const float mn = fmaxf(m, row_max(top)), ms = finite_top(mn);
        if (__builtin_amdgcn_ballot_w64(mn != m)) {
            const float al = exp2_((m - ms) * k.c);
            l *= al;
#pragma unroll
            for (int c = 0; c < PER; ++c) acc[c] *= al;
            m = mn;
        }
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            x[i] = exp2_((x[i] - ms) * k.c);
            l += x[i];
        }
        const typename TL::P p = TL::weights(x);
        // Where some row does not attend to a token that is there, its weight
        // of zero must not meet an infinity or NaN.  Such values are taken out
        // of V, and a row that attends to one gets +inf, -inf or (both, or
        // NaN) their sum in that channel.
        const int j1 = j0 + kTile < len ? j0 + kTile : len;
        if ((j0 < all_lo || j1 > all_hi) && __builtin_amdgcn_ballot_w64(TL::odd(vf))) {
            float in[kVals];
#pragma unroll
            for (int i = 0; i < kVals; ++i) {
                const int j = j0 + TL::key(i, g);
                in[i] = j >= sp.lo && j < sp.hi ? 1.f : 0.f;
            }
            const typename TL::Ones ones = TL::ones(in);
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                const typename TL::Acc up = TL::count_odd(vf, c, TL::kMinusInf, ones);
#pragma unroll
                for (int e = 0; e < TL::kAcc; ++e) acc[c][e] += up[e] > 0.f ? INFINITY : 0.f;
                __builtin_amdgcn_sched_barrier(0);   // a rare path: few registers
                const typename TL::Acc down = TL::count_odd(vf, c, TL::kPlusInf, ones);
#pragma unroll
                for (int e = 0; e < TL::kAcc; ++e) acc[c][e] += down[e] > 0.f ? -INFINITY : 0.f;
                __builtin_amdgcn_sched_barrier(0);
            }
            TL::clear_odd(vf);
        }
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] = TL::pv(vf, c, p, acc[c]);
    };

    // Pages of the next 64 tiles from i0 on, kStep apart, one per lane (of the
    // table's entries past the length too, which block_src leaves out).
    constexpr int kStep = RT == 1 ? kWaves : 1;
    const int cap = a.map.max_pages << a.map.page_shift;
    int pg[kBlocks];
    auto load_pages = [&](int i0) {
        const int j = (tile0 + i0 + kStep * lane) * kTile;
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
            pg[blk] = j + 16 * blk < cap ? page_of(a.map, b, j + 16 * blk) : -1;
    };
    // the cache rows of block blk of tile i, whose pages lane `at` holds (none
    // past the length, on an absent page or past the last tile: such loads
    // give zeros)
    const size_t page_bytes = (size_t)TL::kRowBytes << a.map.page_shift;
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
    if constexpr (RT == 1) {
        // D = 64: two tiles on their way, in two sets of registers.  D = 128: one,
        // as a second set's 64 registers would spill (64 contexts 125 -> 136 us
        // with it; D = 64 in fp32, 8 contexts: 35 -> 31 us).
        constexpr bool kTwo = D == 64;
        struct Ahead {
            typename TL::K kf;
            typename TL::V vf;
            Src src[kBlocks];
        } s0, s1;
        int at = 0;                                 // tiles whose loads have been issued
        auto load_k = [&](Ahead &s) {
            if ((at & 63) == 0) load_pages(w + kWaves * at);
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk)
                s.src[blk] = block_src(w + kWaves * at, at & 63, blk);
            TL::template load_k<STREAM>(s.kf, kc, s.src, a.map.page_shift > 4, lane);
            ++at;
        };
        auto load_v = [&](Ahead &s) {
            rsrc_t rs[kBlocks];
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk)
                rs[blk] = make_rsrc(vc + s.src[blk].at, s.src[blk].bytes);
            TL::template load_v<STREAM>(s.vf, rs, lane);
        };
        auto work = [&](int i, Ahead &s) {
            const int j0 = (tile0 + i) * kTile;
            float x[kVals];
            bool here[kBlocks], full = j0 >= all_lo && j0 + kTile <= all_hi;
            TL::logits(x, s.kf, q);
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) {
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
        for (int i = w; i < tiles; i += kWaves) {
            work(i, s0);
            if constexpr (kTwo) {
                i += kWaves;
                if (i >= tiles) break;
                work(i, s1);
            }
        }
    } else {
        constexpr int kChunks = TL::kRowBytes / 16, kUnits = kTile * kChunks / kThreads;
        static_assert(kUnits * kThreads == kTile * kChunks && 64 / kChunks <= 16,
                      "threads cover a tile, a wave's rows lie in one block of 16");
        // 16 bytes of K and of V per thread, share and unit, and which blocks
        // of this wave's own tile are there
        u32x4 kv[kShares][kUnits][2];
        bool come[kBlocks];
        int paged = 0;                          // the tile that lane 0 of pg stands for
        load_pages(0);
        auto load = [&](int it) {
#pragma unroll
            for (int x = 0; x < kShares; ++x) {
                const int i = it * kShares + x;
                if (i >= paged + 64) {
                    paged = i;
                    load_pages(i);
                }
                Src src[kBlocks];
#pragma unroll
                for (int blk = 0; blk < kBlocks; ++blk) {
                    src[blk] = block_src(i, i - paged, blk);
                    if (x == share) come[blk] = src[blk].bytes != 0;
                }
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const int unit = tid + kThreads * u, row = unit / kChunks;
                    const bool second = uniform(row >> 4) != 0;
                    const size_t at = second ? src[kBlocks - 1].at : src[0].at;
                    const unsigned bytes = second ? src[kBlocks - 1].bytes : src[0].bytes;
                    const unsigned off = (row & 15) * TL::kRowBytes + unit % kChunks * 16;
                    kv[x][u][0] = load16<STREAM>(make_rsrc(kc + at, bytes), off);
                    kv[x][u][1] = load16<STREAM>(make_rsrc(vc + at, bytes), off);
                }
            }
        };
        auto put = [&](char *to, bool (&here)[kBlocks]) {
#pragma unroll
            for (int x = 0; x < kShares; ++x)
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const int unit = tid + kThreads * u;
                    char *p = to + 2 * x * kTileBytes + unit / kChunks * kPitch +
                              unit % kChunks * 16;
                    *reinterpret_cast<u32x4 *>(p) = kv[x][u][0];
                    *reinterpret_cast<u32x4 *>(p + kTileBytes) = kv[x][u][1];
                }
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) here[blk] = come[blk];
        };
        const int its = (tiles + kShares - 1) / kShares;
        bool here[kBlocks];
        load(0);
        put(lds, here);
        __syncthreads();
        for (int it = 0; it < its; ++it) {
            load(it + 1);                       // past the last tile: zeros
            const int j0 = (tile0 + it * kShares + share) * kTile;
            const char *t = lds + (it & 1) * kStage + 2 * share * kTileBytes;
            float x[kVals];
            bool full = j0 >= all_lo && j0 + kTile <= all_hi;
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) full &= here[blk];
            {
                typename TL::K kf;
                TL::lds_k(kf, t, lane);
                TL::logits(x, kf, q);
            }
            typename TL::V vf;
            TL::lds_v(vf, t + kTileBytes, lane);
            absorb(j0, x, vf, full, here);
            put(lds + ((it + 1) & 1) * kStage, here);
            __syncthreads();
        }
    }

    // join the shares: every wave's o in units of the common maximum, summed
    // row by row
    l = row_sum(l);
    if (g == 0) {
        sm[w][r] = m;
        sl[w][r] = l;
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kShares; ++i) top = fmaxf(top, sm[rt + RT * i][r]);
    const float f = exp2_((m - finite_top(top)) * k.c);
    // acc[c][e] is channel dim(c, e, g); those of adjacent c lie together
    constexpr int kRun = PER < 4 ? PER : 4;
    typedef float run_t __attribute__((ext_vector_type(kRun)));
#pragma unroll
    for (int e = 0; e < TL::kAcc; ++e)
#pragma unroll
        for (int c = 0; c < PER; c += kRun) {
            run_t y;
#pragma unroll
            for (int u = 0; u < kRun; ++u) y[u] = acc[c + u][e] * f;
            *reinterpret_cast<run_t *>(&so[w][r][TL::dim(c, e, g)]) = y;
        }
    __syncthreads();
    // 16 threads per row, four channels at a time
#pragma unroll
    for (int i = 0; i < kRows / 16; ++i) {
        const int br = 16 * i + (tid >> 4), orow = row0 + br, ot = br / RW, lr = br % RW;
        if (orow >= rows) break;
        float rtop = -INFINITY, rl = 0.f;
#pragma unroll
        for (int x = 0; x < kShares; ++x) rtop = fmaxf(rtop, sm[ot + RT * x][lr]);
#pragma unroll
        for (int x = 0; x < kShares; ++x)
            rl += sl[ot + RT * x][lr] * exp2_((sm[ot + RT * x][lr] - finite_top(rtop)) * k.c);
        const size_t part = ((size_t)slot * k.plan.units + h * k.plan.row_blocks + rb) * kRows + br;
        const bool alone = sl_.count == 1;
        if ((!alone || k.logits) && (tid & 15) == 0) k.ml[part] = float2{rtop, rl};
        const float inv = 1.f / rl;
        const int t = orow / a.G, hg = orow % a.G;
        T *o = static_cast<T *>(a.o) + (((size_t)b * a.n + t) * a.Hq + h * a.G + hg) * D;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const int d = 64 * u + 4 * (tid & 15);
            f32x4 y = *reinterpret_cast<const f32x4 *>(&so[ot][lr][d]);
#pragma unroll
            for (int x = 1; x < kShares; ++x)
                y += *reinterpret_cast<const f32x4 *>(&so[ot + RT * x][lr][d]);
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
__device__ inline float2 join_ml(const float2 *ml, size_t part, size_t stride, int count, float c) {
    const int lane = threadIdx.x & 63;
    float top = -INFINITY, l = 0.f;
    for (int i = lane; i < count; i += 64) {
        const float2 x = ml[part + i * stride];
        const float mn = fmaxf(top, x.x), ms = finite_top(mn);
        l = l * exp2_((top - ms) * c) + x.y * exp2_((x.x - ms) * c);
        top = mn;
    }
    float all = top;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) all = fmaxf(all, __shfl_xor(all, m));
    all = finite_top(all);
    l *= exp2_((top - all) * c);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) l += __shfl_xor(l, m);
    return float2{all, l};
}

// m, l and four channels of o of some slots.
struct Joined {
    float m, l;
    f32x4 y;
    __device__ inline void add(float mo, float lo, f32x4 yo, float c) {
        const float mn = fmaxf(m, mo), ms = finite_top(mn);
        const float f = exp2_((m - ms) * c), fo = exp2_((mo - ms) * c);
        l = l * f + lo * fo;
        y = y * f + yo * fo;
        m = mn;
    }
};

// Joins the slots' parts, `join_wgs` workgroups per sequence taking its rows
// in turn: D / 4 lanes across a row, the others across slots, a row per wave
// or (many slots) per workgroup.  With scores, further workgroups each add
// the weights of 1,024 tokens of a (sequence, head): a thread sums
// 2^{c (y - m)} / l over the rows, in their order, for four tokens.  These
// cover the table's width, and those past a sequence's length end at once (32
// contexts of up to 6,100 tokens: a call 115 us, 169 under a table of 131,072).
template <typename T, int D, int RW>
__global__ __launch_bounds__(kThreads) void join_kernel(KArgs k, int join_wgs, long long joins,
                                                        long long score_blocks) {
    constexpr int kAcross = D / 4, kGroups = 64 / kAcross;
    const AttnArgs &a = k.a;
    const int tid = threadIdx.x, rows = a.n * a.G;
    const size_t stride = (size_t)k.plan.units * RW;
    if (blockIdx.x < joins) {
        __shared__ __align__(16) Joined other[kWaves][kAcross];
        const int b = (int)(blockIdx.x / join_wgs), part_of = (int)(blockIdx.x % join_wgs);
        const int2 sc = k.sched[b];
        if (sc.y == 1) return;
        const int lane = tid & 63, w = tid >> 6, d = 4 * (lane % kAcross), grp = lane / kAcross;
        const bool together = sc.y > 16;       // four waves to a row
        const int each = together ? kWaves : 1, per = together ? 1 : kWaves;
        for (int q0 = part_of * per; q0 < a.n * a.Hq; q0 += join_wgs * per) {
            const int q = q0 + (together ? 0 : w);
            Joined x{-INFINITY, 0.f, f32x4{0.f, 0.f, 0.f, 0.f}};
            if (q < a.n * a.Hq) {
                const int hq = q % a.Hq, h = hq / a.G, row = q / a.Hq * a.G + hq % a.G;
                const size_t part = (size_t)sc.x * stride +
                                    ((size_t)h * k.plan.row_blocks + row / RW) * RW + row % RW;
#pragma unroll 4
                for (int i = (together ? w : 0) * kGroups + grp; i < sc.y; i += kGroups * each) {
                    const size_t at = part + i * stride;
                    const float2 ml = k.ml[at];
                    x.add(ml.x, ml.y, *reinterpret_cast<const f32x4 *>(k.po + at * D + d), k.c);
                }
            }
#pragma unroll
            for (int m = kAcross; m < 64; m <<= 1)
                x.add(__shfl_xor(x.m, m), __shfl_xor(x.l, m),
                      f32x4{__shfl_xor(x.y.x, m), __shfl_xor(x.y.y, m), __shfl_xor(x.y.z, m),
                            __shfl_xor(x.y.w, m)}, k.c);
            if (together) {
                __syncthreads();               // the last row's have been read
                if (grp == 0) other[w][lane] = x;
                __syncthreads();
                if (w > 0) continue;
#pragma unroll
                for (int i = 1; i < kWaves; ++i) {
                    const Joined o = other[i][lane % kAcross];
                    x.add(o.m, o.l, o.y, k.c);
                }
            }
            if (q < a.n * a.Hq && grp == 0) {
                const float inv = 1.f / x.l;
                f32x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = x.l == 0.f ? 0.f : x.y[e] * inv;
                T *o = static_cast<T *>(a.o) + ((size_t)b * a.n * a.Hq + q) * D + d;
                if constexpr (sizeof(T) == 2) *reinterpret_cast<bf16x4 *>(o) = cvt4(y);
                else                          *reinterpret_cast<f32x4 *>(o) = y;
            }
        }
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
                                    ((size_t)h * k.plan.row_blocks + row / RW) * RW +
                                    row % RW;
                const float2 x = join_ml(k.ml, part, stride, sc.y, k.c);
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
                        if (j + e >= sp.lo && j + e < sp.hi) sum[e] += exp2_((v[e] - st[r].x) * k.c) * st[r].y;
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

template <typename T, int D, int RW, int RT>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    constexpr int kRows = RW * RT;
    const long long cap = (long long)a.map.max_pages << a.map.page_shift;
    const WsMap w = ws_map(a.B, a.n, a.G, a.Hkv, D, kRows, cap, a.scores != nullptr);
    char *ws = static_cast<char *>(a.ws);
    KArgs k{};
    k.a = a;
    k.plan = make_plan(a.B, a.n, a.G, a.Hkv, kRows, cap);
    k.sched = cap > 0 ? reinterpret_cast<int2 *>(ws + w.sched) : nullptr;
    k.ml = reinterpret_cast<float2 *>(ws + w.ml);
    k.po = reinterpret_cast<float *>(ws + w.o);
    k.logits = a.scores && cap > 0 ? reinterpret_cast<float *>(ws + w.logits) : nullptr;
    k.cap32 = (cap + 31) / 32 * 32;
    // (a scale of zero: the smallest number, whose products vanish, as
    // 0 times a masked token's -inf would be NaN; nor is it infinite)
    k.c = fminf(fmaxf(fabsf(a.scale * kLog2e), 1.4e-45f), 3.4e38f);
    k.negative = a.scale < 0.f;
    k.parts = k.plan.max_slots > a.B;
    k.slots = k.parts && a.B > kScan ? reinterpret_cast<int4 *>(ws + w.slots) : nullptr;
    if (k.slots) {
        slots_kernel<<<1, 1024, 0, s>>>(k);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const long long pairs = ((long long)k.plan.max_slots * a.Hkv + 7) / 8 * 8;
    const unsigned grid = (unsigned)(pairs * k.plan.row_blocks);
    if (k.plan.row_blocks == 1) attn_kernel<T, D, RW, RT, true><<<grid, kThreads, 0, s>>>(k);
    else                        attn_kernel<T, D, RW, RT, false><<<grid, kThreads, 0, s>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // about 4,096 workgroups join, and at most one per row: sequences in one
    // slot, often most of them, are left at once
    int join_wgs = a.n * a.Hq;
    const int spread = a.B < 4096 ? 4096 / a.B : 1;
    if (join_wgs > spread) join_wgs = spread;
    const long long joins = k.parts ? (long long)a.B * join_wgs : 0;
    long long score_blocks = a.scores ? (long long)a.B * a.Hkv * ((k.cap32 + 1023) / 1024) : 0;
    if (score_blocks > (1 << 20)) score_blocks = 1 << 20;
    if (joins + score_blocks == 0) return hipSuccess;
    join_kernel<T, D, kRows><<<(unsigned)(joins + score_blocks), kThreads, 0, s>>>(
        k, join_wgs, joins, score_blocks);
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(bool bf16_io, const AttnArgs &a, hipStream_t s) {
    if (!bf16_io) return launch<float, D, 16, 1>(a, s);
    const long long cap = (long long)a.map.max_pages << a.map.page_shift;
    switch (block_rows(true, (long long)a.n * a.G, a.B, a.n, a.Hkv, D, cap, a.window)) {
    case 16: return launch<bf16, D, 16, 1>(a, s);
    case 32: return launch<bf16, D, 32, 1>(a, s);
    default: return launch<bf16, D, 32, 2>(a, s);
    }
}

}  // namespace

size_t attention_workspace(int B, int n, int Hq, int Hkv, int D, long long capacity,
                           bool with_scores) {
    const int G = Hq / Hkv;
    // one size for every dtype and window: the largest over the blocks there can be
    const long long rows = (long long)n * G;
    size_t most = 0;
    for (int rw = 16; rw <= 64 && (rw == 16 || rows > rw / 2); rw *= 2) {
        const size_t x = ws_map(B, n, G, Hkv, D, rw, capacity, with_scores).total;
        if (x > most) most = x;
    }
    return most;
}

hipError_t launch_attention_decode(bool bf16_io, int D, const AttnArgs &a, hipStream_t s) {
    return D == 128 ? launch_d<128>(bf16_io, a, s) : launch_d<64>(bf16_io, a, s);
}

}  // namespace gdr

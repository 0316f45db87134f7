// cache.hip -- the paged key-value cache: writing new tokens, and eviction
// by accumulated attention weight, for gfx950.
#include "cache_internal.h"

namespace gdr {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// What is read once and written once passes through the caches without
// staying there (16 trimmed contexts, 233 MB: 65 -> 60 us).
__device__ inline u32x4 pass_load(const u32x4 *p) { return __builtin_nontemporal_load(p); }
__device__ inline void pass_store(u32x4 *p, u32x4 x) { __builtin_nontemporal_store(x, p); }

// ---------------------------------------------------------------- append
// A copy, bound by bytes (401 MB of prompts, 16 sequences, 8 heads of 128 in
// bf16: 73 us, 5.5 TB/s; a plain copy reaches 5.0): 16 bytes of K and of V per
// thread and unit, kUnits units of a thread in flight together, whose places in
// the cache are found while they are (one unit: 74 us, four: 80, eight: 166).
// Rows are contiguous on both sides: D elements of a token's head, and in the
// cache those of the following tokens behind them.
constexpr int kUnits = 2;
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, int lpr_shift) {
    const unsigned base = blockIdx.x * (256u * kUnits) + threadIdx.x;
    const unsigned units = (unsigned)a.T * a.Hkv << lpr_shift;
    const u32x4 *k = static_cast<const u32x4 *>(a.k), *v = static_cast<const u32x4 *>(a.v);
    u32x4 x[kUnits], y[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const unsigned i = base + 256 * u;
        if (i < units) {
            x[u] = pass_load(k + i);
            y[u] = pass_load(v + i);
        }
    }
    // the sequence of the workgroup's first token: the last b with cu[b] <= t
    int b0 = 0, end = 0;
    if (a.cu_seqlens) {
        const int t0 = (int)((blockIdx.x * (256u * kUnits) >> lpr_shift) / (unsigned)a.Hkv);
        int hi = a.B;
        while (hi - b0 > 1) {
            const int mid = (b0 + hi) >> 1;
            if (a.cu_seqlens[mid] <= t0) b0 = mid; else hi = mid;
        }
        end = a.cu_seqlens[a.B];
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const unsigned i = base + 256 * u, row = i >> lpr_shift;      // (token, head)
        if (i >= units) break;
        const int h = (int)(row % (unsigned)a.Hkv), t = (int)(row / (unsigned)a.Hkv);
        int b = b0;
        long long pos;
        if (a.cu_seqlens) {
            if (t >= end) break;                                      // behind the last sequence
            while (b + 1 < a.B && a.cu_seqlens[b + 1] <= t) ++b;
            pos = (long long)t - a.cu_seqlens[b] + a.start[b];
        } else {
            b = t / a.n_tok;
            pos = (long long)t - (long long)b * a.n_tok + a.start[b];
        }
        if (pos < 0 || pos >= (long long)a.map.max_pages << a.map.page_shift) continue;
        const int page = page_of(a.map, b, (int)pos);
        if (page < 0) continue;
        const size_t cr = cache_row(a.map, a.Hkv, page, h, slot_of(a.map, (int)pos));
        const unsigned c = i & ((1u << lpr_shift) - 1);               // 16 bytes within a row
        pass_store(static_cast<u32x4 *>(a.k_cache) + (cr << lpr_shift) + c, x[u]);
        pass_store(static_cast<u32x4 *>(a.v_cache) + (cr << lpr_shift) + c, y[u]);
        if (a.scores && c == 0) a.scores[cr] = 0.f;
    }
}

// ----------------------------------------------------------------- evict
// Scores as unsigned keys in the same order: absent pages 0, then -inf and
// NaN, ..., -0 and 0 (one key), ..., +inf.
__device__ inline unsigned key_of(float x) {
    if (__builtin_isnan(x)) x = -__builtin_inff();
    const unsigned u = __builtin_bit_cast(unsigned, x == 0.f ? 0.f : x);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Which tokens a (sequence, head) keeps, bound by the latency of its passes:
// 8 us for 600 to 1,000 tokens (8 pairs), 9 us for 1,500 to 4,096 (128 pairs).
// One workgroup per pair, which holds the keys of up to kHeld tokens, read
// once: four adjacent tokens per thread and round, the first eight rounds in
// registers, the others in LDS.  The m-th largest key of the tokens between
// sink and recent is found digit by digit: 8 bits a step, from the top, by a
// histogram of the keys that share the digits found so far, which ends when
// a digit's keys are all wanted.  The kept tokens' places then follow from
// counts over the waves in the tokens' order.  (Longer sequences go through
// the same steps with their keys read anew, kHeld at a time.)
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr int kRegRounds = 8, kRounds = 16;
constexpr int kPerRound = 4 * kSelThreads, kHeld = kRounds * kPerRound;
// Neighbouring scores share their top bits, so that one histogram's counter
// would be hit by most lanes of a wave at once: kCopies of it, in different
// LDS banks, taken by the lanes in turn.
constexpr int kCopies = 16, kCopyStride = 257;

typedef unsigned keys4 __attribute__((ext_vector_type(4)));

// Sum of x over this lane and those below it: shifts by 1, 2, 4 and 8 within
// each 16 lanes, then the sums of 16 and of 32 lanes handed to those above.
__device__ inline int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}
// The digit of the `want`-th largest key: thread t < 256 brings how many keys
// have digit 255 - t.
struct Digit {
    int digit, want, count;                        // wanted of its `count` keys
};
__device__ inline Digit find_digit(int count, int want) {
    __shared__ int waves[4], found[3];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    int incl = count;                              // keys with this digit or a larger one
    if (tid < 256) {
        incl = wave_scan(count);
        if (lane == 63) waves[w] = incl;
    }
    __syncthreads();
    if (tid < 256) {
        for (int i = 0; i < w; ++i) incl += waves[i];
        if (incl >= want && incl - count < want) { // one thread
            found[0] = 255 - tid;
            found[1] = want - (incl - count);
            found[2] = count;
        }
    }
    __syncthreads();
    return Digit{found[0], found[1], found[2]};
}
// Keys that share the digits of `prefix` above `shift` + 8 lie in prefix ..
// prefix + this.
__device__ inline unsigned digit_span(int shift) {
    return shift == 24 ? 0xFFFFFFFFu : (1u << (shift + 8)) - 1;
}
__device__ inline int lanes_below(unsigned long long x) {
    return (int)__builtin_amdgcn_mbcnt_hi((unsigned)(x >> 32),
                                          __builtin_amdgcn_mbcnt_lo((unsigned)x, 0));
}

__device__ inline void select_pair(const EvictArgs &a, int b, int h, int len, int32_t *kept) {
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (len <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < len ? i : -1;
        return;
    }
    const int lo = a.sink, hi = len - a.recent;
    __shared__ int hist[kCopies * kCopyStride];
    __shared__ int2 counts[kRounds][kSelWaves], wave_counts[4];

    __shared__ keys4 lds_keys[(kRounds - kRegRounds) * kSelThreads];
    keys4 reg_keys[kRegRounds];
    auto keys = [&](int r) {
        return r < kRegRounds ? reg_keys[r] : lds_keys[(r - kRegRounds) * kSelThreads + tid];
    };
    // the pages of all rounds, then their scores, eight rounds at a time
    auto load_held = [&](int base) {
        int page[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int j = base + r * kPerRound + 4 * tid;
            page[r] = j < len ? page_of(a.map, b, j) : -1;
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r0 = 0; r0 < kRounds; r0 += 8) {
            if (base + r0 * kPerRound >= len) break;
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // tokens j .. j + 3: one page holds all four
                const int j = base + (r0 + i) * kPerRound + 4 * tid;
                if (page[r0 + i] >= 0)
                    x[i] = *reinterpret_cast<const float4 *>(
                        a.scores + cache_row(a.map, a.Hkv, page[r0 + i], h, slot_of(a.map, j)));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = base + (r0 + i) * kPerRound + 4 * tid;
                keys4 k{0, 0, 0, 0};
                if (page[r0 + i] >= 0) {
                    k = keys4{key_of(x[i].x), key_of(x[i].y), key_of(x[i].z), key_of(x[i].w)};
                    if (j < lo || j + 4 > hi)
#pragma unroll
                        for (int e = 0; e < 4; ++e) k[e] = j + e >= lo && j + e < hi ? k[e] : 0u;
                }
                if (r0 + i < kRegRounds) reg_keys[r0 + i] = k;
                else lds_keys[(r0 + i - kRegRounds) * kSelThreads + tid] = k;
            }
        }
    };
    const bool once = len <= kHeld;
    for (int i = tid; i < kCopies * kCopyStride; i += kSelThreads) hist[i] = 0;
    load_held(0);

    // (Tokens outside lo .. hi have key 0 as well: they add to the count of
    // the digits 00.. only, which comes last and is not compared with.)
    int want = a.budget - a.sink - a.recent;       // of the hi - lo > want tokens between
    unsigned prefix = 0;                           // digits of the threshold found so far
    const bool none = want == 0;
    if (none) prefix = 0xFFFFFFFFu;                // above every key
    bool ties = false;                             // more keys equal the threshold than wanted
    for (int shift = 24; shift >= 0 && !none; shift -= 8) {
        __syncthreads();
        int *mine = hist + (lane & (kCopies - 1)) * kCopyStride;
        const unsigned span = digit_span(shift);
        for (int base = 0; base < len; base += kHeld) {
            if (!once) load_held(base);
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                if (base + r * kPerRound >= len) break;
                const keys4 k4 = keys(r);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k4[e] - prefix <= span) atomicAdd(&mine[(k4[e] >> shift) & 255], 1);
            }
        }
        __syncthreads();
        int count = 0;
        if (tid < 256)
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {        // cleared for the next digit
                count += hist[c * kCopyStride + 255 - tid];
                hist[c * kCopyStride + 255 - tid] = 0;
            }
        const Digit f = find_digit(count, want);
        prefix |= (unsigned)f.digit << shift;
        want = f.want;                             // wanted among the keys with this prefix
        ties = want != f.count;
        if (!ties) break;                          // all of them: prefix 00.. is a threshold
    }
    // Kept are sink and recent, every key above the threshold, and of the
    // keys equal to it the first `want` (without ties: all).
    int above = 0, equal = 0;                      // kept, and equal keys, before base
    for (int base = 0; base < len; base += kHeld) {
        if (!once) load_held(base);
        auto flags = [&](int r, keys4 k, bool (&keep)[4], bool (&eq)[4]) {
            const int j0 = base + r * kPerRound;
            if (j0 >= lo && j0 + kPerRound <= hi && !ties) {      // the usual round
#pragma unroll
                for (int e = 0; e < 4; ++e) { keep[e] = k[e] >= prefix; eq[e] = false; }
                return;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + 4 * tid + e;
                const bool mid = j >= lo && j < hi;
                keep[e] = j < len && (!mid || (ties ? k[e] > prefix : k[e] >= prefix));
                eq[e] = ties && mid && k[e] == prefix;
            }
        };
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (base + r * kPerRound >= len) break;
            bool keep[4], eq[4];
            flags(r, keys(r), keep, eq);
            int2 c{0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c.x += __popcll(__ballot(keep[e]));
                if (ties) c.y += __popcll(__ballot(eq[e]));
            }
            if (lane == 0) counts[r][w] = c;
        }
        __syncthreads();
        // counts before each round and wave: thread t scans entry t, in order
        static_assert(kRounds * kSelWaves == 256, "four waves scan the counts");
        int2 c{0, 0}, t{0, 0};
        if (tid < 256) {
            if (base + (tid / kSelWaves) * kPerRound < len) c = counts[tid / kSelWaves][tid % kSelWaves];
            t = int2{wave_scan(c.x), wave_scan(c.y)};
            if (lane == 63) wave_counts[w] = t;
        }
        __syncthreads();
        if (tid < 256) {
            int2 x{above + t.x - c.x, equal + t.y - c.y};
            for (int i = 0; i < w; ++i) { x.x += wave_counts[i].x; x.y += wave_counts[i].y; }
            counts[tid / kSelWaves][tid % kSelWaves] = x;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) { above += wave_counts[i].x; equal += wave_counts[i].y; }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (base + r * kPerRound >= len) break;
            int nk = counts[r][w].x, ne = counts[r][w].y;
            // before this lane's four tokens
            bool keep[4], eq[4];
            flags(r, keys(r), keep, eq);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                nk += lanes_below(__ballot(keep[e]));
                if (ties) ne += lanes_below(__ballot(eq[e]));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (keep[e] || (eq[e] && ne < want))
                    kept[nk + (ne < want ? ne : want)] = base + r * kPerRound + 4 * tid + e;
                nk += keep[e];
                ne += eq[e];
            }
        }
    }
}

// The places of row i of the new order and of the row it comes from, as rows
// of the caches; false where it is not moved.
__device__ inline bool row_move(const EvictArgs &a, int b, int h, int i, int j, size_t &src,
                                size_t &dst) {
    const int from = page_of(a.map, b, j), to = page_of(a.to, b, i);
    src = cache_row(a.map, a.Hkv, from, h, slot_of(a.map, j));
    dst = cache_row(a.to, a.Hkv, to, h, slot_of(a.to, i));
    return from >= 0 && to >= 0;
}
constexpr int kMoveRows = 4;       // rows of a thread, their loads in flight together

// Rows base .. of a pair's first m, 16 bytes of K and of V per thread and row,
// kMoveRows of THREADS / (row's threads) rows, every row on its own.
template <int THREADS>
__device__ inline void move_rows(const EvictArgs &a, int b, int h, int base, int m, int lpr_shift,
                                 const int32_t *kept) {
    const int tid = threadIdx.x, c = tid & ((1 << lpr_shift) - 1), rows = THREADS >> lpr_shift;
    u32x4 *kc = static_cast<u32x4 *>(a.k_cache), *vc = static_cast<u32x4 *>(a.v_cache);
    size_t src[kMoveRows], dst[kMoveRows];
    bool move[kMoveRows];
    u32x4 x[kMoveRows], y[kMoveRows];
    float sc[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
        const int i = base + rows * u + (tid >> lpr_shift);
        move[u] = i < m && row_move(a, b, h, i, kept[i < m ? i : 0], src[u], dst[u]);
    }
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
        if (move[u]) {
            x[u] = pass_load(kc + (src[u] << lpr_shift) + c);
            y[u] = pass_load(vc + (src[u] << lpr_shift) + c);
            if (c == 0) sc[u] = a.scores[src[u]];
        }
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
        if (move[u]) {
            pass_store(kc + (dst[u] << lpr_shift) + c, x[u]);
            pass_store(vc + (dst[u] << lpr_shift) + c, y[u]);
            if (c == 0) a.scores[dst[u]] = sc[u];
        }
}

// MOVE: the kept rows go into the new pages here as well, which saves a launch
// where a pair's rows are few: 128 KiB of K and V each, 8 pairs 12.5 -> 11.5 us,
// 256 pairs 21.3 -> 19.9; 32 KiB, 1,024 pairs 41 -> 38.  With more to move one
// workgroup per pair is too few (256 KiB, 8 pairs: 12.2 -> 14.9 us).
constexpr int kMoveBytes = 128 << 10;
template <bool MOVE>
__global__ __launch_bounds__(kSelThreads) void select_kernel(EvictArgs a, int lpr_shift) {
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    const int len = cached_len(a.seq_lens, b, a.map);
    int32_t *kept = a.kept + (size_t)blockIdx.x * a.budget;
    select_pair(a, b, h, len, kept);
    if constexpr (MOVE) {
        const int m = len < a.budget ? len : a.budget;
        if (h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
        __syncthreads();                               // all of kept is there
        for (int base = 0; base < m; base += (kSelThreads >> lpr_shift) * kMoveRows)
            move_rows<kSelThreads>(a, b, h, base, m, lpr_shift, kept);
    }
}

// The same for few (sequence, head) pairs with long sequences: one workgroup
// reads a pair's scores at some 20 GB/s, so each pair is given `chunks`
// workgroups of `chunk` tokens.  A launch per digit: every workgroup finds the
// last digit from all chunks' histograms (each writes its own), adds up which of
// its keys that puts above the threshold, and makes its histogram of the next
// digit; the last launch places the chunk's kept tokens behind those of the
// chunks before it.  (65,001 tokens, 8 heads: 53 us by one workgroup, 28 us so,
// the five launches' 4.0, 6.0, 5.8, 5.6 and 7.5.)  The lengths are on the device:
// short sequences under a table past kSpreadTokens take this way too (8 pairs of
// 600 to 1,000 tokens, a whole call 25 us; 11.5 under a table up to that).
constexpr int kSpreadPairs = 64;       // at most so many pairs ...
constexpr int kSpreadTokens = 8192;    // ... and tables longer than this
constexpr int kSpreadChunks = 64;
struct Spread {
    int chunks, chunk;         // chunk: a multiple of kPerRound
    int *hist;                 // [4 digits][pairs][chunks][256]
    int *above;                // [pairs][chunks]: keys above the threshold's digits so far
    int4 *state;               // [5][pairs]: prefix, want, done, ties before each launch
};
struct SpreadLayout {
    int chunks, chunk;
    size_t above, state, total;
};
SpreadLayout spread_layout(int pairs, long long capacity) {
    SpreadLayout l{};
    if (pairs > kSpreadPairs || capacity <= kSpreadTokens) return l;
    const long long c = (capacity + kSpreadChunks - 1) / kSpreadChunks;
    l.chunk = (int)((c + kPerRound - 1) / kPerRound * kPerRound);
    l.chunks = (int)((capacity + l.chunk - 1) / l.chunk);
    const size_t cells = (size_t)pairs * l.chunks;
    l.above = cells * 4 * 256 * sizeof(int);
    l.state = l.above + (cells * sizeof(int) + 255) / 256 * 256;
    l.total = l.state + (size_t)pairs * 5 * sizeof(int4);
    return l;
}

__global__ __launch_bounds__(kSelThreads) void spread_kernel(EvictArgs a, Spread s, int level) {
    // a pair's chunks stay on one XCD when the pairs are a multiple of eight
    // (workgroups go to the eight in turn), and with them their histograms in
    // its L2: the whole call 61 -> 57 us
    const int pairs = a.B * a.Hkv, pair = blockIdx.x % pairs, me = blockIdx.x / pairs;
    const int b = pair / a.Hkv, h = pair % a.Hkv, tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int len = cached_len(a.seq_lens, b, a.map);
    int32_t *kept = a.kept + (size_t)pair * a.budget;
    if (len <= a.budget) {
        if (level == 4)
            for (int i = me * kSelThreads + tid; i < a.budget; i += s.chunks * kSelThreads)
                kept[i] = i < len ? i : -1;
        return;
    }
    const int lo = a.sink, hi = len - a.recent, t0 = me * s.chunk;
    if (t0 >= len) return;
    const int t1 = t0 + s.chunk < len ? t0 + s.chunk : len;
    const int used = (len + s.chunk - 1) / s.chunk;      // chunks with tokens
    auto cell = [&](int digit, int c) {
        return s.hist + (((size_t)digit * pairs + pair) * s.chunks + c) * 256;
    };
    __shared__ int hist[kCopies * kCopyStride], sums[3];
    __shared__ int2 counts[kSelWaves];
    // the threshold so far: its digits, the keys wanted among those that share
    // them, whether it is found, and whether more keys equal it than wanted
    unsigned prefix = 0;
    int want = a.budget - a.sink - a.recent;
    bool done = want == 0, ties = false;
    if (done) prefix = 0xFFFFFFFFu;                      // above every key
    // keys above it, and equal to it, in the chunks before this one (level 4)
    int above = 0, equal = 0;
    if (level > 0) {
        const int4 st = s.state[(size_t)(level - 1) * pairs + pair];
        prefix = (unsigned)st.x; want = st.y; done = st.z != 0; ties = st.w != 0;
        if (tid < 3) sums[tid] = 0;
        __syncthreads();
        if (level == 4 && tid < me) atomicAdd(&sums[0], s.above[(size_t)pair * s.chunks + tid]);
        if (!done) {
            // four groups of 256 threads take the chunks in turn
            const int digit = 255 - (tid & 255), grp = tid >> 8;
            int part = 0;
#pragma unroll 8
            for (int c = grp; c < used; c += 4) part += cell(level - 1, c)[digit];
            if (tid < 256) hist[digit] = 0;
            __syncthreads();
            if (part) atomicAdd(&hist[digit], part);
            __syncthreads();
            const Digit f = find_digit(tid < 256 ? hist[digit] : 0, want);
            prefix |= (unsigned)f.digit << (32 - 8 * level);
            want = f.want;
            ties = want != f.count;
            done = !ties || level == 4;
            // own keys (level 4: those of the chunks before) above the digit, and with it
            if (digit >= f.digit) {
                int n = 0;
                if (level == 4) {
#pragma unroll 8
                    for (int c = grp; c < me; c += 4) n += cell(3, c)[digit];
                } else if (grp == 0) {
                    n = cell(level - 1, me)[digit];
                }
                if (n) atomicAdd(&sums[digit == f.digit ? 2 : 1], n);
            }
        }
        __syncthreads();
        if (level == 4) {
            above = sums[0] + sums[1] + (ties ? 0 : sums[2]);
            equal = ties ? sums[2] : 0;
        } else if (tid == 0) {
            int *x = s.above + (size_t)pair * s.chunks + me;
            const int old = level == 1 ? 0 : *x;
            *x = old + sums[1] + (done ? sums[2] : 0);   // without ties the equal ones are kept
        }
    }
    if (me == 0 && tid == 0 && level < 4)
        s.state[(size_t)level * pairs + pair] = int4{(int)prefix, want, done, ties};
    if (level < 4 && done) return;

    auto load4 = [&](int j) {
        keys4 k{0, 0, 0, 0};
        const int page = j < len ? page_of(a.map, b, j) : -1;
        if (page >= 0) {
            const float4 x = *reinterpret_cast<const float4 *>(
                a.scores + cache_row(a.map, a.Hkv, page, h, slot_of(a.map, j)));
            k = keys4{key_of(x.x), key_of(x.y), key_of(x.z), key_of(x.w)};
            if (j < lo || j + 4 > hi)
#pragma unroll
                for (int e = 0; e < 4; ++e) k[e] = j + e >= lo && j + e < hi ? k[e] : 0u;
        }
        return k;
    };
    if (level < 4) {
        const int shift = 24 - 8 * level;
        const unsigned span = digit_span(shift);
        for (int i = tid; i < kCopies * kCopyStride; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        int *mine = hist + (lane & (kCopies - 1)) * kCopyStride;
        for (int base = t0; base < t1; base += kPerRound) {
            const int j = base + 4 * tid;
            const bool inside = j >= lo && j + 4 <= hi;
            const keys4 k = load4(j);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k[e] - prefix <= span && (inside || (j + e >= lo && j + e < hi)))
                    atomicAdd(&mine[(k[e] >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid < 256) {
            int count = 0;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) count += hist[c * kCopyStride + 255 - tid];
            cell(level, me)[255 - tid] = count;
        }
        return;
    }
    // sink and recent tokens before this chunk
    above += (t0 < lo ? t0 : lo) + (t0 > hi ? t0 - hi : 0);
    for (int base = t0; base < t1; base += kPerRound) {
        const keys4 k = load4(base + 4 * tid);
        bool keep[4], eq[4];
        int2 c{0, 0}, before{0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = base + 4 * tid + e;
            const bool mid = j >= lo && j < hi;
            keep[e] = j < len && (!mid || (ties ? k[e] > prefix : k[e] >= prefix));
            eq[e] = ties && mid && k[e] == prefix;
            const unsigned long long bk = __ballot(keep[e]), be = __ballot(eq[e]);
            before.x += lanes_below(bk);
            before.y += lanes_below(be);
            c.x += __popcll(bk);
            c.y += __popcll(be);
        }
        __syncthreads();
        if (lane == 0) counts[w] = c;
        __syncthreads();
        int nk = above + before.x, ne = equal + before.y;
#pragma unroll
        for (int i = 0; i < kSelWaves; ++i) {
            const int2 x = counts[i];
            nk += i < w ? x.x : 0;
            ne += i < w ? x.y : 0;
            above += x.x;
            equal += x.y;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (keep[e] || (eq[e] && ne < want)) kept[nk + (ne < want ? ne : want)] = base + 4 * tid + e;
            nk += keep[e];
            ne += eq[e];
        }
    }
}

// Rows kept[b, h, i] -> i into other pages.  A copy, bound by bytes: 16
// contexts trimmed to 1,800 tokens (8 heads of 128, bf16), 233 MB in 48 us, 4.8
// TB/s.
__global__ __launch_bounds__(256) void copy_rows_kernel(EvictArgs a, int lpr_shift) {
    const int pair = blockIdx.x, b = pair / a.Hkv, h = pair % a.Hkv;
    const int len = cached_len(a.seq_lens, b, a.map);
    const int m = len < a.budget ? len : a.budget;
    if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
    const int tile = (256 >> lpr_shift) * kMoveRows;
    for (int base = blockIdx.y * tile; base < m; base += gridDim.y * tile)
        move_rows<256>(a, b, h, base, m, lpr_shift, a.kept + (size_t)pair * a.budget);
}

constexpr int kCloseRows = 4;

// The same in place: a workgroup has a column of the rows of one (sequence,
// head), of K (even blockIdx.y) or V, 16 << slice_shift bytes wide, and goes
// through the rows in order, a tile of them read, then written.  kept[i] >= i
// and kept ascends, so that a
// tile's writes lie at or below its own reads and below all later ones, and
// the next tile can be read before this one is written.  Columns are 64 bytes
// wide, or 16 where the pairs are too few to fill the card (16,384 tokens kept
// of 8 heads, this kernel alone: 149 us at 64, 80 us at 16; copied into other
// pages 29 us.  128 pairs of 1,800: 57 us, copied 48).
__global__ __launch_bounds__(256) void close_up_kernel(EvictArgs a, int lpr_shift,
                                                       int slice_shift) {
    const int across = 256 >> slice_shift, tile_rows = across * kCloseRows;
    const int pair = blockIdx.x, b = pair / a.Hkv, h = pair % a.Hkv, tid = threadIdx.x;
    const int lane = tid & ((1 << slice_shift) - 1), c = ((blockIdx.y >> 1) << slice_shift) + lane;
    const int len = cached_len(a.seq_lens, b, a.map);
    const int m = len < a.budget ? len : a.budget;
    // (new_lens may be seq_lens: what another workgroup has written gives the
    // same m)
    if (blockIdx.y == 0 && h == 0 && tid == 0) a.new_lens[b] = m;
    const int32_t *kept = a.kept + (size_t)pair * a.budget;
    u32x4 *cache = static_cast<u32x4 *>(blockIdx.y & 1 ? a.v_cache : a.k_cache);
    const bool scores = blockIdx.y == 0 && lane == 0;
    struct Tile {
        size_t dst[kCloseRows];
        bool move[kCloseRows];
        u32x4 x[kCloseRows];
        float sc[kCloseRows];
    };
    auto load = [&](int base, Tile &t) {
        size_t src[kCloseRows];
#pragma unroll
        for (int u = 0; u < kCloseRows; ++u) {
            const int i = base + across * u + (tid >> slice_shift), j = i < m ? kept[i] : i;
            t.move[u] = i != j && row_move(a, b, h, i, j, src[u], t.dst[u]);
        }
#pragma unroll
        for (int u = 0; u < kCloseRows; ++u)
            if (t.move[u]) {
                t.x[u] = cache[(src[u] << lpr_shift) + c];
                if (scores) t.sc[u] = a.scores[src[u]];
            }
    };
    Tile t;
    load(0, t);
    for (int base = 0; base < m; base += tile_rows) {
        // the tile is read (vmcnt(0)) by every wave before any of it is written
        __builtin_amdgcn_s_waitcnt(0x0f70);
        __syncthreads();
        Tile next;
        load(base + tile_rows, next);
#pragma unroll
        for (int u = 0; u < kCloseRows; ++u)
            if (t.move[u]) {
                cache[(t.dst[u] << lpr_shift) + c] = t.x[u];
                if (scores) a.scores[t.dst[u]] = t.sc[u];
            }
        t = next;
    }
}

int lpr_shift_of(int row_bytes) { return row_bytes == 128 ? 3 : row_bytes == 256 ? 4 : 5; }

}  // namespace

hipError_t launch_cache_append(int row_bytes, const AppendArgs &a, hipStream_t s) {
    const int sh = lpr_shift_of(row_bytes);
    const long long units = (long long)a.T * a.Hkv << sh;
    append_kernel<<<(unsigned)((units + 256 * kUnits - 1) / (256 * kUnits)), 256, 0, s>>>(a, sh);
    return hipGetLastError();
}

size_t evict_workspace(int pairs, long long capacity) {
    return spread_layout(pairs, capacity).total;
}

hipError_t launch_cache_evict(int row_bytes, const EvictArgs &a, hipStream_t s) {
    const int sh = lpr_shift_of(row_bytes);
    const int pairs = a.B * a.Hkv;
    const long long capacity = (long long)a.map.max_pages << a.map.page_shift;
    const SpreadLayout l = spread_layout(pairs, capacity);
    if (l.chunks) {
        char *ws = static_cast<char *>(a.ws);
        const Spread sp{l.chunks, l.chunk, reinterpret_cast<int *>(ws),
                        reinterpret_cast<int *>(ws + l.above), reinterpret_cast<int4 *>(ws + l.state)};
        for (int level = 0; level <= 4; ++level) {
            spread_kernel<<<pairs * l.chunks, kSelThreads, 0, s>>>(a, sp, level);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    } else {
        // (new lengths written over the old ones would be read as such by the
        // other heads' workgroups)
        const bool apart = a.new_lens + a.B <= a.seq_lens || a.seq_lens + a.B <= a.new_lens;
        const bool move = !a.in_place && apart && (long long)a.budget * row_bytes * 2 <= kMoveBytes;
        if (move) select_kernel<true><<<pairs, kSelThreads, 0, s>>>(a, sh);
        else      select_kernel<false><<<pairs, kSelThreads, 0, s>>>(a, sh);
        const hipError_t e = hipGetLastError();
        if (move || e != hipSuccess) return e;
    }
    if (a.in_place) {
        const int slice = pairs * (2 << (sh - 2)) >= 256 ? 2 : 0;
        close_up_kernel<<<dim3(pairs, 2 << (sh - slice)), 256, 0, s>>>(a, sh, slice);
    } else {
        const int most = a.budget < capacity ? a.budget : (int)capacity;
        const int tile = (256 >> sh) * kMoveRows;
        int tiles = (most + tile - 1) / tile;
        tiles = tiles < 1 ? 1 : (tiles > 16384 ? 16384 : tiles);
        copy_rows_kernel<<<dim3(pairs, tiles), 256, 0, s>>>(a, sh);
    }
    return hipGetLastError();
}

}  // namespace gdr

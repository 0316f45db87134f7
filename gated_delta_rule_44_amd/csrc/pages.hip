// pages.hip -- the paged cache's bookkeeping on the GPU, for gfx950: the tokens
// kept of a tree of drafts, and page tables that follow the sequences' lengths.
#include "cache_internal.h"
#include "device_util.h"
#include "wave.h"

namespace gdr {
namespace {

// ------------------------------------------------------------------ accept

// What is kept of one sequence's drafts: those on the way to the leaf that
// have a place, one bit each, and where they go.
struct Kept {
    unsigned long long drafts;
    int from, to;                // places of draft 0 and of the first kept one
};
// By one wave.  The way up takes a scalar step a draft.
__device__ inline Kept kept_drafts(const AcceptArgs &a, int b) {
    const int u = threadIdx.x & 63;
    int up = u < a.n ? a.parents[(size_t)b * a.n + u] : -1;
    int at = uniform(a.leaf[b]);
    const int len = uniform(cached_len(a.seq_lens, b, a.map));
    if (up >= u) up = -1;
    if (at >= a.n) at = -1;
    Kept k{0, len - a.n, len > a.n ? len - a.n : 0};
    while (at >= 0) {
        k.drafts |= 1ull << at;
        at = __builtin_amdgcn_readlane(up, at);
    }
    if (k.from < 0) k.drafts &= k.from <= -64 ? 0 : ~0ull << -k.from;
    return k;
}
__device__ inline void write_end(const AcceptArgs &a, int b, const Kept &k) {
    const int u = threadIdx.x & 63, count = __builtin_popcountll(k.drafts);
    const int rank = __builtin_popcountll(k.drafts & ((1ull << u) - 1));
    if (k.drafts >> u & 1) a.path[(size_t)b * a.n + rank] = u;
    if (u >= count && u < a.n) a.path[(size_t)b * a.n + u] = -1;
    if (u == 0) a.new_lens[b] = k.to + count;
}

// Workgroup = (sequence, head).  A kept draft's place is never behind the one
// it goes to, so that rows taken in their order, some at a time, can be moved
// in place: a pass reads all of its rows before it writes one, and no later
// one reads what it wrote.  Latency bounds it, of the way up, the page numbers and
// the rows, one after the other: 1.7 us for 7 drafts of one request, 4.2 for 64
// requests of 24 (8 heads of 128 in bf16, with scores: 6.3 MB, 1.3 us at a copy's
// rate).
constexpr int kMoveThreads = 256, kUnits = 4;
template <int ROW_BYTES>
__global__ __launch_bounds__(kMoveThreads) void accept_kernel(AcceptArgs a) {
    constexpr int kChunks = ROW_BYTES / 16;                 // 16 bytes of K and of V each
    constexpr int kPass = kMoveThreads * kUnits / kChunks;  // rows of a pass
    __shared__ int path[64];
    const int tid = threadIdx.x, b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    const Kept k = kept_drafts(a, b);
    if (tid < 64) {
        if (a.ends && h == 0) write_end(a, b, k);
        if (k.drafts >> tid & 1) path[__builtin_popcountll(k.drafts & ((1ull << tid) - 1))] = tid;
    }
    __syncthreads();
    const int count = __builtin_popcountll(k.drafts);
    // the cache rows of kept draft i, or false if it stays
    auto rows_of = [&](int i, size_t &from, size_t &to) {
        if (i >= count) return false;
        const int j = k.from + path[i], d = k.to + i;
        if (j == d) return false;
        const int pj = page_of(a.map, b, j), pd = page_of(a.map, b, d);
        if (pj < 0 || pd < 0) return false;
        from = cache_row(a.map, a.Hkv, pj, h, slot_of(a.map, j));
        to = cache_row(a.map, a.Hkv, pd, h, slot_of(a.map, d));
        return true;
    };
    for (int i0 = 0; i0 < count; i0 += kPass) {
        u32x4 kv[kUnits][2];
        size_t to[kUnits], from;
        bool some[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int unit = tid + kMoveThreads * u, c = unit % kChunks;
            some[u] = rows_of(i0 + unit / kChunks, from, to[u]);
            if (some[u]) {
                const size_t at = from * kChunks + c;
                kv[u][0] = static_cast<const u32x4 *>(a.k_cache)[at];
                kv[u][1] = static_cast<const u32x4 *>(a.v_cache)[at];
                to[u] = to[u] * kChunks + c;
            }
        }
        float score = 0.f;
        size_t score_to = 0;
        bool scored = false;
        if (a.scores && tid < kPass) {
            scored = rows_of(i0 + tid, from, score_to);
            if (scored) score = a.scores[from];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            if (some[u]) {
                static_cast<u32x4 *>(a.k_cache)[to[u]] = kv[u][0];
                static_cast<u32x4 *>(a.v_cache)[to[u]] = kv[u][1];
            }
        if (scored) a.scores[score_to] = score;
    }
}

// New lengths that overwrite the old ones, once every head has read these: a
// wave per sequence.
__global__ __launch_bounds__(64) void accept_end_kernel(AcceptArgs a) {
    write_end(a, blockIdx.x, kept_drafts(a, blockIdx.x));
}

template <int ROW_BYTES>
hipError_t accept(const AcceptArgs &a, hipStream_t s) {
    AcceptArgs x = a;
    x.ends = a.new_lens != a.seq_lens;
    accept_kernel<ROW_BYTES><<<(unsigned)(a.B * a.Hkv), kMoveThreads, 0, s>>>(x);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || x.ends) return e;
    accept_end_kernel<<<(unsigned)a.B, 64, 0, s>>>(x);
    return hipGetLastError();
}

// ------------------------------------------------------------------ resize

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kGroup = 16;                       // words of a group of pages
constexpr int kWords = kMaxPages / 32, kGroups = kWords / kGroup;
constexpr int kRowsAtOnce = 16;                  // rows whose entries a wave requests together

// Sums over the workgroup's threads before this one; total: over all.
__device__ inline int scan(int x, int &total, int *lds) {
    const int w = threadIdx.x >> 6, incl = wave_scan(x);
    if ((threadIdx.x & 63) == 63) lds[w] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const int v = lds[i];
        before += i < w ? v : 0;
        total += v;
    }
    __syncthreads();
    return before + incl - x;
}

// One workgroup does all, as each step needs the whole of the one before: the
// pages that some row keeps, as bits in LDS; how many are free in the groups of
// 512 before each; and, 1,024 rows at a time, which rows are served, from the
// sums of what they ask for, and the new entries, a thread each, whatever rows
// they are of.  An entry's page is the free one of its number: a search over the
// groups' sums, then within one group.  Latency bounds it (256 rows of up to 128
// pages: 9 us, 4 rows 4.6).
__global__ __launch_bounds__(kThreads) void resize_kernel(ResizeArgs a) {
    __shared__ __align__(16) unsigned used[kWords];
    __shared__ int free_before[kGroups];
    __shared__ int keeps[kThreads], have[kThreads], first[kThreads];
    __shared__ int sums[kWaves], given;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int groups = (a.num_pages + 32 * kGroup - 1) / (32 * kGroup), words = groups * kGroup;
    const long long cap = (long long)a.max_pages * a.page_size;
    const int shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz(a.page_size) : -1;
    auto pages = [&](int tokens) {
        const long long n = (long long)tokens + a.page_size - 1;
        return (int)(shift >= 0 ? n >> shift : n / a.page_size);
    };
    // a row's lengths, in tokens and in pages
    int old = 0, now = 0, x = 0, y = 0;
    auto load = [&](int b) {
        old = now = x = y = 0;
        if (b < a.B) {
            const int l = a.seq_lens[b], m = a.want[b];
            old = (int)(l < 0 ? 0 : (l > cap ? cap : l));
            now = (int)(m < 0 ? 0 : (m > cap ? cap : m));
            x = pages(old);
            y = pages(now);
        }
    };
    for (int i = tid; i < words; i += kThreads) {
        const int left = a.num_pages - 32 * i;            // bits past the last page are taken
        used[i] = left >= 32 ? 0u : (left <= 0 ? ~0u : ~0u << left);
    }
    if (tid == 0) given = 0;
    for (int row0 = 0; row0 < a.B; row0 += kThreads) {
        load(row0 + tid);
        keeps[tid] = x < y ? x : y;
        __syncthreads();
        for (int r0 = w * kRowsAtOnce; r0 < kThreads && row0 + r0 < a.B; r0 += kWaves * kRowsAtOnce) {
            // (a lane's row's entries, and the longest of the 16)
            int keep[kRowsAtOnce], longest = 0;
#pragma unroll
            for (int u = 0; u < kRowsAtOnce; ++u) {
                keep[u] = keeps[r0 + u];
                longest = keep[u] > longest ? keep[u] : longest;
            }
            const int32_t *rows = a.table + (size_t)(row0 + r0) * a.max_pages;
            for (int c0 = 0; c0 < longest; c0 += 64) {
                const int c = c0 + lane;
                int page[kRowsAtOnce];
#pragma unroll
                for (int u = 0; u < kRowsAtOnce; ++u)
                    page[u] = c < keep[u] ? rows[(size_t)u * a.max_pages + c] : -1;
#pragma unroll
                for (int u = 0; u < kRowsAtOnce; ++u)
                    if ((unsigned)page[u] < (unsigned)a.num_pages)
                        atomicOr(&used[page[u] >> 5], 1u << (page[u] & 31));
            }
        }
        __syncthreads();
    }
    __syncthreads();
    int free_all = 0;
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
        int n = 0, total;
        if (g0 + tid < groups) {
            const u32x4 *word = reinterpret_cast<const u32x4 *>(used + (g0 + tid) * kGroup);
#pragma unroll
            for (int i = 0; i < kGroup / 4; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) n += __builtin_popcount(~word[i][u]);
        }
        const int before = scan(n, total, sums);
        if (g0 + tid < groups) free_before[g0 + tid] = free_all + before;
        free_all += total;
    }
    // the free page of number k < free_all
    auto free_page = [&](int k) {
        int lo = 0, n = groups;                           // the last group with free_before <= k
        while (n > 1) {
            const int half = n / 2;
            const bool up = free_before[lo + half] <= k;
            lo = up ? lo + half : lo;
            n = up ? n - half : half;
        }
        k -= free_before[lo];
        const u32x4 *group = reinterpret_cast<const u32x4 *>(used + lo * kGroup);
        unsigned word = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const unsigned f = ~group[i / 4][i % 4];
            const int c = __builtin_popcount(f);
            if (k >= 0 && k < c) {
                word = f;
                at = i | k << 8;
            }
            k -= c;
        }
        int bit = 0, left = at >> 8;
        at &= 255;
#pragma unroll
        for (int half = 16; half; half >>= 1) {
            const int c = __builtin_popcount(word >> bit & ((1u << half) - 1));
            if (left >= c) {
                left -= c;
                bit += half;
            }
        }
        return 32 * (lo * kGroup + at) + bit;
    };
    int asked = 0, grown = 0, done = 0;
    for (int row0 = 0; row0 < a.B; row0 += kThreads) {
        const int b = row0 + tid;
        if (a.B > kThreads) load(b);
        // (a row that asks for more than there are is not served, nor any after
        // it: sums of 1,024 such numbers are below 2^31)
        int all, more = y > x ? y - x : 0;
        more = more > a.num_pages ? a.num_pages + 1 : more;
        const int before = asked + scan(more, all, sums);
        asked = asked + all < 1 << 29 ? asked + all : 1 << 29;
        // what is asked for only grows, so that every row served before this one
        // got all that was asked for up to it
        const bool served = more == 0 || (before <= free_all && before + more <= free_all);
        if (!served) {
            now = old;
            y = x;
        }
        have[tid] = x;
        first[tid] = before;
        if (served && more) atomicMax(&given, before + more);
        const int up = scan(now > old ? now - old : 0, all, sums);    // (and LDS is written)
        if (b < a.B) {
            a.new_lens[b] = now;
            if (a.cu_seqlens) a.cu_seqlens[b] = grown + up;
        }
        grown += all;
        // the new entries, whose numbers are their free pages': of the last row
        // that starts at or before a number
        const int end = given;
        for (int n = done + tid; n < end; n += kThreads) {
            int r = 0;
#pragma unroll
            for (int half = kThreads / 2; half; half >>= 1) r = first[r + half] <= n ? r + half : r;
            a.table[(size_t)(row0 + r) * a.max_pages + have[r] + n - first[r]] = free_page(n);
        }
        done = end;
        // the dropped ones, a wave's rows in turn
        unsigned long long drops = __builtin_amdgcn_ballot_w64(x > y);
        while (drops) {
            const int u = __builtin_ctzll(drops);
            drops &= drops - 1;
            const int from = __builtin_amdgcn_readlane(y, u), to = __builtin_amdgcn_readlane(x, u);
            int32_t *row = a.table + (size_t)(row0 + 64 * w + u) * a.max_pages;
            for (int c = from + lane; c < to; c += 64) row[c] = -1;
        }
        __syncthreads();
    }
    if (tid == 0) {
        if (a.cu_seqlens) a.cu_seqlens[a.B] = grown;
        if (a.free_pages) a.free_pages[0] = free_all - done;
    }
}

}  // namespace

hipError_t launch_cache_accept(int row_bytes, const AcceptArgs &a, hipStream_t s) {
    switch (row_bytes) {
    case 128: return accept<128>(a, s);
    case 256: return accept<256>(a, s);
    default:  return accept<512>(a, s);
    }
}

hipError_t launch_cache_resize(const ResizeArgs &a, hipStream_t s) {
    resize_kernel<<<1, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gdr

// pages.hip -- the paged cache's bookkeeping on the GPU, for gfx950: the tokens
// kept of a tree of drafts, and page tables that follow the sequences' lengths.
#include "cache_internal.h"
#include "device_util.h"

namespace gdr {
namespace {

__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

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
// one reads what it wrote.
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
constexpr int kRowsAtOnce = 8;                   // rows whose entries a wave requests together

// Sums over the workgroup's threads before this one; total: over all.
__device__ inline long long scan(long long x, long long &total, long long *lds) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    long long incl = x;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const long long y = __shfl_up(incl, m);
        if (lane >= m) incl += y;
    }
    if (lane == 63) lds[w] = incl;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const long long v = lds[i];
        before += i < w ? v : 0;
        total += v;
    }
    __syncthreads();
    return before + incl - x;
}

// One workgroup does all, as each step needs the whole of the one before: the
// pages that some row keeps, as bits in LDS; how many are free in the groups of
// 512 before each; and, 1,024 rows at a time, which rows are served, from the
// sums of what they ask for, and their entries.  An entry's page is the free
// one of its number: a search over the groups' sums, then within one group.
__global__ __launch_bounds__(kThreads) void resize_kernel(ResizeArgs a) {
    __shared__ __align__(16) unsigned used[kWords];
    __shared__ int free_before[kGroups];
    __shared__ int have[kThreads], need[kThreads], first[kThreads];
    __shared__ long long sums[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int groups = (a.num_pages + 32 * kGroup - 1) / (32 * kGroup), words = groups * kGroup;
    const long long cap = (long long)a.max_pages * a.page_size;
    auto held = [&](const int32_t *lens, int b) {
        const int l = lens[b];
        return (int)(l < 0 ? 0 : (l > cap ? cap : l));
    };
    auto pages = [&](int tokens) {
        return (int)(((long long)tokens + a.page_size - 1) / a.page_size);
    };
    for (int i = tid; i < words; i += kThreads) {
        const int left = a.num_pages - 32 * i;            // bits past the last page are taken
        used[i] = left >= 32 ? 0u : (left <= 0 ? ~0u : ~0u << left);
    }
    // entries of the rows from row0 on, lo .. hi of each, a wave's rows together
    auto entries = [&](int row0, const int *lo, const int *hi, auto &&f) {
        for (int r0 = w * kRowsAtOnce; r0 < kThreads && row0 + r0 < a.B; r0 += kWaves * kRowsAtOnce) {
            int longest = 0;
#pragma unroll
            for (int u = 0; u < kRowsAtOnce; ++u) {
                const int n = hi[r0 + u] - (lo ? lo[r0 + u] : 0);
                longest = n > longest ? n : longest;
            }
            for (int c = lane; c < longest + lane; c += 64) f(r0, c);
        }
    };
    for (int row0 = 0; row0 < a.B; row0 += kThreads) {
        const int b = row0 + tid;
        int keep = 0;
        if (b < a.B) {
            const int x = pages(held(a.seq_lens, b)), y = pages(held(a.want, b));
            keep = x < y ? x : y;
        }
        have[tid] = keep;
        __syncthreads();
        entries(row0, nullptr, have, [&](int r0, int c) {
            int page[kRowsAtOnce];
#pragma unroll
            for (int u = 0; u < kRowsAtOnce; ++u)
                page[u] = c < have[r0 + u]
                              ? a.table[(size_t)(row0 + r0 + u) * a.max_pages + c] : -1;
#pragma unroll
            for (int u = 0; u < kRowsAtOnce; ++u)
                if ((unsigned)page[u] < (unsigned)a.num_pages)
                    atomicOr(&used[page[u] >> 5], 1u << (page[u] & 31));
        });
        __syncthreads();
    }
    __syncthreads();
    int free_all = 0;
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
        int n = 0;
        if (g0 + tid < groups) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) n += __builtin_popcount(~used[(g0 + tid) * kGroup + i]);
        }
        long long total;
        const int before = (int)scan(n, total, sums);
        if (g0 + tid < groups) free_before[g0 + tid] = free_all + before;
        free_all += (int)total;
    }
    __syncthreads();
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
        unsigned word = 0;
        int at = 0, seen = 0;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const unsigned x = ~used[lo * kGroup + i];
            const int c = __builtin_popcount(x);
            if (seen <= k && k < seen + c) {
                word = x;
                at = i;
                k -= seen;
                seen = 1 << 30;
            }
            seen += c;
        }
        int bit = 0;
#pragma unroll
        for (int half = 16; half; half >>= 1) {
            const int c = __builtin_popcount(word >> bit & ((1u << half) - 1));
            if (k >= c) {
                k -= c;
                bit += half;
            }
        }
        return 32 * (lo * kGroup + at) + bit;
    };
    long long asked = 0, grown = 0;
    int given = 0;
    for (int row0 = 0; row0 < a.B; row0 += kThreads) {
        const int b = row0 + tid;
        int old = 0, now = 0, x = 0, y = 0;
        if (b < a.B) {
            old = held(a.seq_lens, b);
            now = held(a.want, b);
            x = pages(old);
            y = pages(now);
        }
        const int more = y > x ? y - x : 0;
        long long all;
        const long long before = asked + scan(more, all, sums);
        asked += all;
        // what is asked for only grows, so that every row served before this one
        // got all that was asked for up to it
        const bool served = more == 0 || before + more <= free_all;
        if (!served) {
            now = old;
            y = x;
        }
        have[tid] = x;
        need[tid] = y;
        first[tid] = served && more ? (int)before : 0;
        const long long up = scan(now > old ? now - old : 0, all, sums);
        if (b < a.B) {
            a.new_lens[b] = now;
            if (a.cu_seqlens) a.cu_seqlens[b] = (int)(grown + up);
        }
        grown += all;
        scan(served ? more : 0, all, sums);               // (and have, need, first are there)
        given += (int)all;
        // columns past the shorter of the two lengths: new pages, or none
        for (int r = w; r < kThreads && row0 + r < a.B; r += kWaves) {
            const int x = have[r], y = need[r];
            int32_t *row = a.table + (size_t)(row0 + r) * a.max_pages;
            for (int c = x + lane; c < y; c += 64) row[c] = free_page(first[r] + c - x);
            for (int c = y + lane; c < x; c += 64) row[c] = -1;
        }
        __syncthreads();
    }
    if (tid == 0) {
        if (a.cu_seqlens) a.cu_seqlens[a.B] = (int)grown;
        if (a.free_pages) a.free_pages[0] = free_all - given;
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

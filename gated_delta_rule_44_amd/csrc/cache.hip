// cache.hip -- the paged key-value cache: writing new tokens, and eviction
// by accumulated attention weight, for gfx950.
#include "cache_internal.h"

namespace gdr {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- append
// One thread per 16 bytes of a token's rows, for K and V both.
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, int lpr_shift) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(i & ((1 << lpr_shift) - 1));          // 16 bytes within a row
    const long long row = i >> lpr_shift;                     // (token, head)
    const int h = (int)(row % a.Hkv);
    const long long t = row / a.Hkv;
    if (t >= a.T) return;
    int b;
    long long pos;
    if (a.cu_seqlens) {
        if (t >= a.cu_seqlens[a.B]) return;                   // behind the last sequence
        int lo = 0, hi = a.B;                                 // the last b with cu[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
        }
        b = lo;
        pos = t - a.cu_seqlens[b] + a.start[b];
    } else {
        b = (int)(t / a.n_tok);
        pos = t - (long long)b * a.n_tok + a.start[b];
    }
    if (pos < 0 || pos >= (long long)a.map.max_pages << a.map.page_shift) return;
    const int page = page_of(a.map, b, (int)pos);
    if (page < 0) return;
    const size_t cr = cache_row(a.map, a.Hkv, page, h, slot_of(a.map, (int)pos));
    const size_t dst = (cr << lpr_shift) + c;
    static_cast<u32x4 *>(a.k_cache)[dst] = static_cast<const u32x4 *>(a.k)[i];
    static_cast<u32x4 *>(a.v_cache)[dst] = static_cast<const u32x4 *>(a.v)[i];
    if (a.scores && c == 0) a.scores[cr] = 0.f;
}

// ----------------------------------------------------------------- evict
// Scores as unsigned keys in the same order: absent pages 0, then -inf and
// NaN, ..., -0 and 0 (one key), ..., +inf.
__device__ inline unsigned key_of(float x) {
    if (__builtin_isnan(x)) x = -__builtin_inff();
    const unsigned u = __builtin_bit_cast(unsigned, x == 0.f ? 0.f : x);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ inline unsigned key_at(const EvictArgs &a, int b, int h, int j) {
    const int page = page_of(a.map, b, j);
    return page < 0 ? 0u : key_of(a.scores[cache_row(a.map, a.Hkv, page, h, slot_of(a.map, j))]);
}

constexpr int kSelThreads = 1024;

// Sum of x over the workgroup's threads before this one, and over all.
__device__ inline int block_scan(int x, int &total, int *lds) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int incl = x;
    for (int m = 1; m < 64; m <<= 1) {
        const int y = __shfl_up(incl, m);
        if (lane >= m) incl += y;
    }
    if (lane == 63) lds[w] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < kSelThreads / 64; ++i) {
        const int v = lds[i];
        before += i < w ? v : 0;
        total += v;
    }
    __syncthreads();
    return before + incl - x;
}

// Which tokens a (sequence, head) keeps: one workgroup per pair.  The m-th
// largest key of the tokens between sink and recent is found digit by digit
// (8 bits, from the top, by histograms of the keys that share the digits
// found so far); a last pass in the tokens' order writes the kept ones.
__global__ __launch_bounds__(kSelThreads) void select_kernel(EvictArgs a) {
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x;
    const int len = cached_len(a.seq_lens, b, a.map);
    int32_t *kept = a.kept + (size_t)blockIdx.x * a.budget;
    if (len <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < len ? i : -1;
        return;
    }
    const int lo = a.sink, hi = len - a.recent;
    int want = a.budget - a.sink - a.recent;       // of hi - lo > want tokens
    __shared__ int hist[256], found[2], scan[kSelThreads / 64];
    unsigned prefix = 0;                           // digits of the threshold found so far
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = lo + tid; j < hi; j += kSelThreads) {
            const unsigned k = key_at(a, b, h, j);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int d = 255, left = want;
            while (hist[d] < left) left -= hist[d--];
            found[0] = d;
            found[1] = left;
        }
        __syncthreads();
        prefix |= (unsigned)found[0] << shift;
        want = found[1];                           // wanted among the keys with this prefix
        __syncthreads();
    }
    // every key above prefix is kept, and the first `want` keys equal to it
    const bool none = a.budget == a.sink + a.recent;
    int above = 0, equal = 0;                      // kept, and equal keys, before this chunk
    for (int base = 0; base < len; base += kSelThreads) {
        const int j = base + tid;
        int keep = 0, eq = 0;
        if (j < len) {
            if (j < lo || j >= hi) {
                keep = 1;
            } else if (!none) {
                const unsigned k = key_at(a, b, h, j);
                keep = k > prefix;
                eq = k == prefix;
            }
        }
        int tot_k, tot_e;
        const int bk = block_scan(keep, tot_k, scan), be = block_scan(eq, tot_e, scan);
        const int e = equal + be;
        if (keep || (eq && e < want)) kept[above + bk + (e < want ? e : want)] = j;
        above += tot_k;
        equal += tot_e;
    }
}

// Rows kept[b, h, i] -> i, one workgroup per (sequence, head) and 16 bytes
// of the rows.  In place, a tile of rows is read, then written: kept[i] >= i
// and kept ascends, so a tile's writes lie below everything the later tiles
// read.
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a, int lpr_shift) {
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, c = blockIdx.y, tid = threadIdx.x;
    const int len = cached_len(a.seq_lens, b, a.map);
    const int m = len < a.budget ? len : a.budget;
    const int32_t *kept = a.kept + (size_t)blockIdx.x * a.budget;
    u32x4 *kc = static_cast<u32x4 *>(a.k_cache), *vc = static_cast<u32x4 *>(a.v_cache);
    for (int base = 0; base < m; base += 256) {
        const int i = base + tid;
        u32x4 x, y;
        float sc = 0.f;
        size_t dst = 0;
        bool move = false;
        if (i < m) {
            const int j = kept[i];
            const int from = page_of(a.map, b, j), to = page_of(a.to, b, i);
            move = from >= 0 && to >= 0 && !(a.in_place && i == j);
            if (move) {
                const size_t src = cache_row(a.map, a.Hkv, from, h, slot_of(a.map, j));
                dst = cache_row(a.to, a.Hkv, to, h, slot_of(a.to, i));
                x = kc[(src << lpr_shift) + c];
                y = vc[(src << lpr_shift) + c];
                if (c == 0) sc = a.scores[src];
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): the tile is read ...
        __syncthreads();                      // ... by every wave before any writes
        if (move) {
            kc[(dst << lpr_shift) + c] = x;
            vc[(dst << lpr_shift) + c] = y;
            if (c == 0) a.scores[dst] = sc;
        }
    }
    if (h == 0 && c == 0 && tid == 0) a.new_lens[b] = m;
}

int lpr_shift_of(int row_bytes) { return row_bytes == 128 ? 3 : row_bytes == 256 ? 4 : 5; }

}  // namespace

hipError_t launch_cache_append(int row_bytes, const AppendArgs &a, hipStream_t s) {
    const int sh = lpr_shift_of(row_bytes);
    const long long units = (long long)a.T * a.Hkv << sh;
    append_kernel<<<(unsigned)((units + 255) / 256), 256, 0, s>>>(a, sh);
    return hipGetLastError();
}

hipError_t launch_cache_evict(int row_bytes, const EvictArgs &a, hipStream_t s) {
    const int sh = lpr_shift_of(row_bytes);
    select_kernel<<<a.B * a.Hkv, kSelThreads, 0, s>>>(a);
    move_kernel<<<dim3(a.B * a.Hkv, 1 << sh), 256, 0, s>>>(a, sh);
    return hipGetLastError();
}

}  // namespace gdr

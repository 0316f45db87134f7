// cache_internal.h -- shared declarations of the paged cache's kernels and
// their host side.  Internal to the library: the public interface is
// include/gdr_cache.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

// Where the tokens are.  An entry of `table` outside 0..pages-1 marks an
// absent page.
struct PageMap {
    const int32_t *table;    // [B, max_pages]
    int max_pages;
    int page_shift;          // log2 of page_size, 4..8
    int pages;               // pages in the caches
};

// The page of token j of sequence b, or -1 if absent; 0 <= j < capacity.
__device__ inline int page_of(const PageMap &m, int b, int j) {
    const int p = m.table[(size_t)b * m.max_pages + (j >> m.page_shift)];
    return (unsigned)p < (unsigned)m.pages ? p : -1;
}
__device__ inline int slot_of(const PageMap &m, int j) {
    return j & ((1 << m.page_shift) - 1);
}
// Row (page, head, slot) of a cache: the index of its first element is this
// times D (64 bits: a cache may hold more than 2^32 elements).
__device__ inline size_t cache_row(const PageMap &m, int Hkv, int page, int h, int slot) {
    return (((size_t)page * Hkv + h) << m.page_shift) + slot;
}
// A sequence's length, brought into 0..capacity.
__device__ inline int cached_len(const int32_t *seq_lens, int b, const PageMap &m) {
    const int cap = m.max_pages << m.page_shift;
    const int l = seq_lens[b];
    return l < 0 ? 0 : (l > cap ? cap : l);
}

struct AppendArgs {
    const void *k, *v;           // [T, Hkv, D]
    const int32_t *cu_seqlens;   // [B+1] or nullptr (n_tok each)
    const int32_t *start;        // [B]
    PageMap map;
    void *k_cache, *v_cache;     // [pages, Hkv, page, D]
    float *scores;               // [pages, Hkv, page] or nullptr
    int B, n_tok, T, Hkv;
};
hipError_t launch_cache_append(int row_bytes, const AppendArgs &a, hipStream_t s);

struct AttnArgs {
    const void *q;               // [B, n, Hq, D]
    const void *k_cache, *v_cache;
    PageMap map;
    const int32_t *seq_lens;     // [B]
    float *scores;               // [pages, Hkv, page] or nullptr
    void *o;                     // [B, n, Hq, D]
    void *ws;
    int B, n, Hq, Hkv, G;        // G = Hq / Hkv
    float scale;
    int window;                  // 0: none
    const int32_t *parents;      // [B, n]: a tree of drafts; nullptr: a chain
};
// of a decode, or of a tree as well
size_t attention_workspace(int B, int n, int Hq, int Hkv, int D, long long capacity,
                           bool with_scores, bool tree);
hipError_t launch_attention_decode(bool bf16_io, int D, const AttnArgs &a, hipStream_t s);
// drafts of a tree (a.parents), 64 of a sequence at most; no scores
hipError_t launch_attention_tree(bool bf16_io, int D, const AttnArgs &a, hipStream_t s);

struct EvictArgs {
    void *k_cache, *v_cache;
    float *scores;
    PageMap map, to;             // to: where the kept tokens go (== map: in place)
    bool in_place;
    const int32_t *seq_lens;     // [B]
    int32_t *new_lens;           // [B]
    int32_t *kept;               // [B, Hkv, budget]
    void *ws;
    int B, Hkv, budget, recent, sink;
};
size_t evict_workspace(int pairs, long long capacity);
hipError_t launch_cache_evict(int row_bytes, const EvictArgs &a, hipStream_t s);

struct AcceptArgs {
    void *k_cache, *v_cache;
    float *scores;               // or nullptr
    PageMap map;
    const int32_t *seq_lens;     // [B]
    const int32_t *parents;      // [B, n]
    const int32_t *leaf;         // [B]
    int32_t *new_lens;           // [B]
    int32_t *path;               // [B, n]
    int B, n, Hkv;
    bool ends;                   // the moves' launch writes new_lens and path as well
};
hipError_t launch_cache_accept(int row_bytes, const AcceptArgs &a, hipStream_t s);

constexpr int kMaxPages = 1 << 20;   // of a resize
struct ResizeArgs {
    int32_t *table;              // [B, max_pages]
    const int32_t *seq_lens, *want;
    int32_t *new_lens;           // [B]
    int32_t *cu_seqlens;         // [B+1] or nullptr
    int32_t *free_pages;         // [1] or nullptr
    int B, max_pages, page_size, num_pages;
};
hipError_t launch_cache_resize(const ResizeArgs &a, hipStream_t s);

}  // namespace gdr

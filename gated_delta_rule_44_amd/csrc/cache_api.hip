// cache_api.hip -- the C ABI declared in include/gdr_cache.h: host-side
// argument checks and launches on the caller's stream.  Every check runs
// before the first HIP call, so a rejected call has no side effects.  No C++
// exception crosses the interface.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/gdr_cache.h"
#include "api_util.h"
#include "cache_internal.h"

namespace {

using gdr::aligned16;
using gdr::check_workspace;
using gdr::fail;
using gdr::finish;

// A launch holds fewer than 2^32 threads: rows of new tokens (up to 32
// threads each), query rows (256 threads), trimmed pairs (1,024 threads)
constexpr long long kMaxRows = 1LL << 26, kMaxQueryRows = 1LL << 23, kMaxPairs = 1LL << 21;

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

#define REQUIRE_I32(p, name)                                                       \
    do {                                                                           \
        if (!(p)) return fail(GDR_EINVAL, "%s: %s is NULL", what, name);           \
        if (!aligned4(p)) return fail(GDR_EINVAL, "%s: %s is not 4-byte aligned",  \
                                      what, name);                                 \
    } while (0)

// a * b * c >= limit, for non-negative factors whose product may not fit
bool reaches(long long a, long long b, long long c, long long limit) {
    return (__int128)a * b * c >= limit;
}

// the log2 of a supported page size, or -1
int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// dtype, width, heads and the cache's geometry
gdr_status check_cache(const char *what, int dt, int B, int Hkv, int D, int max_pages,
                       int page_size, int num_pages) {
    if (dt != GDR_F32 && dt != GDR_BF16)
        return fail(GDR_EINVAL, "%s: dtype %d is not GDR_F32 or GDR_BF16", what, dt);
    if (D != 64 && D != 128)
        return fail(GDR_EUNSUPPORTED, "%s: D = %d; supported widths are 64 and 128", what, D);
    if (B < 0 || Hkv <= 0 || max_pages < 0 || num_pages < 0)
        return fail(GDR_EINVAL, "%s: bad sizes B=%d Hkv=%d max_pages=%d num_pages=%d", what, B,
                    Hkv, max_pages, num_pages);
    if (page_shift_of(page_size) < 0)
        return fail(GDR_EUNSUPPORTED,
                    "%s: page_size = %d; supported sizes are 16, 32, 64, 128 and 256", what,
                    page_size);
    if ((long long)max_pages * page_size >= (1LL << 30))
        return fail(GDR_EUNSUPPORTED, "%s: a table of %d pages of %d tokens is too long", what,
                    max_pages, page_size);
    if ((long long)num_pages * Hkv >= (1LL << 31))
        return fail(GDR_EUNSUPPORTED, "%s: %d pages x %d heads is too large", what, num_pages, Hkv);
    return GDR_OK;
}

// A host copy of a page table: every entry in -1..num_pages-1, and none
// twice where `once` is not NULL (num_pages flags, kept over several tables).
gdr_status check_table(const char *what, const char *name, const int32_t *t, int B, int max_pages,
                       int num_pages, unsigned char *once) {
    const long long n = (long long)B * max_pages;
    for (long long i = 0; i < n; ++i) {
        if (t[i] < -1 || t[i] >= num_pages)
            return fail(GDR_EINVAL, "%s: %s[%lld, %lld] = %d outside -1..%d", what, name,
                        i / max_pages, i % max_pages, t[i], num_pages - 1);
        if (once && t[i] >= 0) {
            if (once[t[i]])
                return fail(GDR_EINVAL, "%s: page %d is in %s twice, or in both tables", what,
                            t[i], name);
            once[t[i]] = 1;
        }
    }
    return GDR_OK;
}

}  // namespace

extern "C" {

gdr_status gdr_cache_append(enum gdr_dtype dt, int B, int n_tok, int T_total, int Hkv, int D,
                            const void *k, const void *v, const int32_t *cu_seqlens,
                            const int32_t *cu_seqlens_host, const int32_t *start,
                            const int32_t *page_table, int max_pages, int page_size,
                            int num_pages, void *k_cache, void *v_cache, float *scores,
                            void *stream) {
    const char *what = "gdr_cache_append";
    gdr_status st = check_cache(what, dt, B, Hkv, D, max_pages, page_size, num_pages);
    if (st != GDR_OK) return st;
    if (n_tok < 0 || T_total < 0)
        return fail(GDR_EINVAL, "%s: bad sizes n_tok=%d T_total=%d", what, n_tok, T_total);
    if (!cu_seqlens && (long long)B * n_tok != T_total)
        return fail(GDR_EINVAL, "%s: T_total = %d but B * n_tok = %lld", what, T_total,
                    (long long)B * n_tok);
    // one thread per 16 bytes of a row, in a grid of less than 2^32 threads
    if ((long long)T_total * Hkv >= kMaxRows)
        return fail(GDR_EUNSUPPORTED, "%s: %lld rows exceed %lld", what, (long long)T_total * Hkv,
                    kMaxRows);
    if (cu_seqlens_host) {
        if (!cu_seqlens)
            return fail(GDR_EINVAL, "%s: cu_seqlens_host given without cu_seqlens", what);
        if (cu_seqlens_host[0] != 0)
            return fail(GDR_EINVAL, "%s: cu_seqlens[0] = %d, expected 0", what, cu_seqlens_host[0]);
        for (int i = 0; i < B; ++i)
            if (cu_seqlens_host[i + 1] < cu_seqlens_host[i])
                return fail(GDR_EINVAL, "%s: cu_seqlens decreases at %d", what, i);
        if (cu_seqlens_host[B] > T_total)
            return fail(GDR_EINVAL, "%s: cu_seqlens[B] = %d but T_total = %d", what,
                        cu_seqlens_host[B], T_total);
    }
    if (B == 0 || T_total == 0 || max_pages == 0 || num_pages == 0) return GDR_OK;
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(v, "v");
    if (cu_seqlens) REQUIRE_I32(cu_seqlens, "cu_seqlens");
    REQUIRE_I32(start, "start");
    REQUIRE_I32(page_table, "page_table");
    REQUIRE_PTR(k_cache, "k_cache");
    REQUIRE_PTR(v_cache, "v_cache");
    REQUIRE_ALIGNED_OR_NULL(scores, "scores");
    gdr::AppendArgs a{};
    a.k = k; a.v = v; a.cu_seqlens = cu_seqlens; a.start = start;
    a.map = gdr::PageMap{page_table, max_pages, page_shift_of(page_size), num_pages};
    a.k_cache = k_cache; a.v_cache = v_cache; a.scores = scores;
    a.B = B; a.n_tok = n_tok; a.T = T_total; a.Hkv = Hkv;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_cache_append(D * (dt == GDR_BF16 ? 2 : 4), a, s), s, what);
}

size_t gdr_attention_workspace_bytes(int B, int n_tok, int Hq, int Hkv, int D, int max_pages,
                                     int page_size, int with_scores) {
    if (B <= 0 || n_tok <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || D <= 0 || max_pages < 0 ||
        page_shift_of(page_size) < 0 || (long long)max_pages * page_size >= (1LL << 30) ||
        reaches(B, n_tok, Hq, kMaxQueryRows))
        return 0;
    return gdr::attention_workspace(B, n_tok, Hq, Hkv, D, (long long)max_pages * page_size,
                                    with_scores != 0);
}

gdr_status gdr_attention_decode(enum gdr_dtype dt, int B, int n_tok, int Hq, int Hkv, int D,
                                float scale, int window, const void *q, const void *k_cache,
                                const void *v_cache, const int32_t *page_table,
                                const int32_t *page_table_host, int max_pages, int page_size,
                                int num_pages, const int32_t *seq_lens, float *scores, void *o,
                                void *workspace, size_t ws_bytes, void *stream) {
    const char *what = "gdr_attention_decode";
    gdr_status st = check_cache(what, dt, B, Hkv, D, max_pages, page_size, num_pages);
    if (st != GDR_OK) return st;
    if (n_tok < 0 || Hq <= 0)
        return fail(GDR_EINVAL, "%s: bad sizes n_tok=%d Hq=%d", what, n_tok, Hq);
    if (Hq % Hkv)
        return fail(GDR_EINVAL, "%s: Hq (%d) is not a multiple of Hkv (%d)", what, Hq, Hkv);
    if (!isfinite(scale)) return fail(GDR_EINVAL, "%s: scale is not finite", what);
    if (window < 0) return fail(GDR_EINVAL, "%s: window = %d; 0 means none", what, window);
    if (reaches(B, n_tok, Hq, kMaxQueryRows))
        return fail(GDR_EUNSUPPORTED, "%s: %d x %d x %d query rows exceed %lld", what, B, n_tok, Hq,
                    kMaxQueryRows);
    if (page_table_host) {
        unsigned char *once = nullptr;
        if (scores) {
            once = static_cast<unsigned char *>(calloc(num_pages > 0 ? num_pages : 1, 1));
            if (!once) return fail(GDR_EINVAL, "%s: host memory for the page check", what);
        }
        st = check_table(what, "page_table", page_table_host, B, max_pages, num_pages, once);
        free(once);
        if (st != GDR_OK) return st;
    }
    if (B == 0 || n_tok == 0) return GDR_OK;
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(o, "o");
    REQUIRE_I32(seq_lens, "seq_lens");
    if (max_pages > 0) REQUIRE_I32(page_table, "page_table");
    if (num_pages > 0) {
        REQUIRE_PTR(k_cache, "k_cache");
        REQUIRE_PTR(v_cache, "v_cache");
    }
    REQUIRE_ALIGNED_OR_NULL(scores, "scores");
    st = check_workspace(what, workspace, ws_bytes,
                         gdr_attention_workspace_bytes(B, n_tok, Hq, Hkv, D, max_pages, page_size,
                                                       scores != nullptr));
    if (st != GDR_OK) return st;
    gdr::AttnArgs a{};
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    // without pages every token is absent: the kernels see empty sequences
    a.map = gdr::PageMap{page_table, num_pages > 0 ? max_pages : 0, page_shift_of(page_size),
                         num_pages};
    a.seq_lens = seq_lens; a.scores = scores; a.o = o; a.ws = workspace;
    a.B = B; a.n = n_tok; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
    a.scale = scale; a.window = window;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_attention_decode(dt == GDR_BF16, D, a, s), s, what);
}

size_t gdr_cache_evict_workspace_bytes(int B, int Hkv, int max_pages, int page_size) {
    if (B <= 0 || Hkv <= 0 || max_pages <= 0 || page_shift_of(page_size) < 0 ||
        (long long)B * Hkv >= kMaxPairs || (long long)max_pages * page_size >= (1LL << 30))
        return 0;
    return gdr::evict_workspace(B * Hkv, (long long)max_pages * page_size);
}

gdr_status gdr_cache_evict(enum gdr_dtype dt, int B, int Hkv, int D, int budget, int recent,
                           int sink, void *k_cache, void *v_cache, float *scores,
                           const int32_t *page_table, const int32_t *page_table_host,
                           int max_pages, const int32_t *new_page_table,
                           const int32_t *new_page_table_host, int new_max_pages,
                           int page_size, int num_pages, const int32_t *seq_lens,
                           int32_t *new_lens, int32_t *kept, void *workspace, size_t ws_bytes,
                           void *stream) {
    const char *what = "gdr_cache_evict";
    gdr_status st = check_cache(what, dt, B, Hkv, D, max_pages, page_size, num_pages);
    if (st != GDR_OK) return st;
    if (budget < 1 || recent < 0 || sink < 0 || (long long)recent + sink > budget)
        return fail(GDR_EINVAL, "%s: budget=%d recent=%d sink=%d; sink + recent must fit the budget",
                    what, budget, recent, sink);
    if (budget >= (1 << 30))
        return fail(GDR_EUNSUPPORTED, "%s: budget = %d is too large", what, budget);
    if ((long long)B * Hkv >= kMaxPairs)
        return fail(GDR_EUNSUPPORTED, "%s: %lld (sequence, head) pairs exceed %lld", what,
                    (long long)B * Hkv, kMaxPairs);
    if (!new_page_table && new_page_table_host)
        return fail(GDR_EINVAL, "%s: new_page_table_host given without new_page_table", what);
    if (new_page_table) {
        const long long cap = (long long)max_pages * page_size;
        const long long need = budget < cap ? budget : cap;
        if (new_max_pages < 0 || (long long)new_max_pages * page_size < need ||
            (long long)new_max_pages * page_size >= (1LL << 30))
            return fail(GDR_EINVAL, "%s: a new table of %d pages of %d tokens for %lld tokens", what,
                        new_max_pages, page_size, need);
    }
    if (page_table_host || new_page_table_host) {
        unsigned char *once =
            static_cast<unsigned char *>(calloc(num_pages > 0 ? num_pages : 1, 1));
        if (!once) return fail(GDR_EINVAL, "%s: host memory for the page check", what);
        // the pages the call writes first, each once; then the pages it only
        // reads, which may be shared but not written
        if (new_page_table_host)
            st = check_table(what, "new_page_table", new_page_table_host, B, new_max_pages,
                             num_pages, once);
        if (st == GDR_OK && page_table_host) {
            if (!new_page_table) {
                st = check_table(what, "page_table", page_table_host, B, max_pages, num_pages, once);
            } else {
                st = check_table(what, "page_table", page_table_host, B, max_pages, num_pages,
                                 nullptr);
                const long long n = (long long)B * max_pages;
                for (long long i = 0; st == GDR_OK && i < n; ++i)
                    if (page_table_host[i] >= 0 && once[page_table_host[i]])
                        st = fail(GDR_EINVAL, "%s: page %d is in both tables", what,
                                  page_table_host[i]);
            }
        }
        free(once);
        if (st != GDR_OK) return st;
    }
    if (B == 0) return GDR_OK;
    REQUIRE_I32(seq_lens, "seq_lens");
    REQUIRE_I32(new_lens, "new_lens");
    REQUIRE_I32(kept, "kept");
    if (max_pages > 0) REQUIRE_I32(page_table, "page_table");
    if (new_page_table) REQUIRE_I32(new_page_table, "new_page_table");
    if (num_pages > 0) {
        REQUIRE_PTR(k_cache, "k_cache");
        REQUIRE_PTR(v_cache, "v_cache");
        REQUIRE_PTR(scores, "scores");
    }
    st = check_workspace(what, workspace, ws_bytes,
                         gdr_cache_evict_workspace_bytes(B, Hkv, max_pages, page_size));
    if (st != GDR_OK) return st;
    gdr::EvictArgs a{};
    a.ws = workspace;
    a.k_cache = k_cache; a.v_cache = v_cache; a.scores = scores;
    const int shift = page_shift_of(page_size);
    a.map = gdr::PageMap{page_table, max_pages, shift, num_pages};
    a.in_place = new_page_table == nullptr;
    a.to = a.in_place ? a.map : gdr::PageMap{new_page_table, new_max_pages, shift, num_pages};
    a.seq_lens = seq_lens; a.new_lens = new_lens; a.kept = kept;
    a.B = B; a.Hkv = Hkv; a.budget = budget; a.recent = recent; a.sink = sink;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_cache_evict(D * (dt == GDR_BF16 ? 2 : 4), a, s), s, what);
}

}  // extern "C"

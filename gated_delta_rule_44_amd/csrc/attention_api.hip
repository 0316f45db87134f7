// attention_api.hip -- the C ABI declared in include/gdr_attention.h: host-side
// argument checks and launches on the caller's stream.  Every check runs
// before the first HIP call, so a rejected call has no side effects.  No C++
// exception crosses the interface.
#include <math.h>

#include "../../include/gdr_attention.h"
#include "api_util.h"
#include "cache_check.h"
#include "cache_internal.h"
#include "prompt_internal.h"

namespace {

using gdr::aligned16;
using gdr::aligned4;
using gdr::check_cache;
using gdr::check_table;
using gdr::check_workspace;
using gdr::fail;
using gdr::finish;
using gdr::kMaxDrafts;
using gdr::kMaxPairs;
using gdr::kMaxQueryRows;
using gdr::page_shift_of;
using gdr::reaches;

gdr_status check_heads(const char *what, int dt, int Hq, int Hkv, int D, float scale, int window) {
    if (dt != GDR_F32 && dt != GDR_BF16)
        return fail(GDR_EINVAL, "%s: dtype %d is not GDR_F32 or GDR_BF16", what, dt);
    if (D != 64 && D != 128)
        return fail(GDR_EUNSUPPORTED, "%s: D = %d; supported widths are 64 and 128", what, D);
    if (Hq <= 0 || Hkv <= 0) return fail(GDR_EINVAL, "%s: bad sizes Hq=%d Hkv=%d", what, Hq, Hkv);
    if (Hq % Hkv)
        return fail(GDR_EINVAL, "%s: Hq (%d) is not a multiple of Hkv (%d)", what, Hq, Hkv);
    if (!isfinite(scale)) return fail(GDR_EINVAL, "%s: scale is not finite", what);
    if (window < 0) return fail(GDR_EINVAL, "%s: window = %d; 0 means none", what, window);
    return GDR_OK;
}

// sizes and offsets of a batch of prompts
gdr_status check_prompts(const char *what, int dt, int B, int T, int T_total, int Hq, int Hkv, int D,
                         float scale, int window, const int32_t *cu_seqlens,
                         const int32_t *cu_seqlens_host) {
    const gdr_status st = check_heads(what, dt, Hq, Hkv, D, scale, window);
    if (st != GDR_OK) return st;
    if (B < 0 || T < 0 || T_total < 0)
        return fail(GDR_EINVAL, "%s: bad sizes B=%d T=%d T_total=%d", what, B, T, T_total);
    if (!cu_seqlens && (long long)B * T != T_total)
        return fail(GDR_EINVAL, "%s: T_total = %d but B * T = %lld", what, T_total,
                    (long long)B * T);
    if ((long long)Hq * D > (1 << 20))
        return fail(GDR_EUNSUPPORTED, "%s: %d heads of %d are too wide", what, Hq, D);
    // a launch holds fewer than 2^32 threads: 256 for 64 rows of a head (the
    // least of the long forms), and a sequence may leave one block unused; a row
    // and a window add up to a 32-bit number
    if (T_total >= (1 << 29) || ((long long)T_total / 64 + B) * Hq >= (1LL << 24))
        return fail(GDR_EUNSUPPORTED, "%s: %d rows in %d sequences of %d heads are too many", what,
                    T_total, B, Hq);
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
    return GDR_OK;
}

// offsets that are not looked at
const int32_t kAnyOffsets[1] = {0};

gdr::PromptArgs prompt_args(int B, int T, int T_total, int Hq, int Hkv, float scale, int window,
                            const void *q, const void *k, const void *v, const int32_t *cu_seqlens) {
    gdr::PromptArgs a{};
    a.q = q; a.k = k; a.v = v; a.cu = cu_seqlens;
    a.B = B; a.T = T; a.T_total = T_total; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
    a.scale = scale;
    // (a window as wide as the sequences is none)
    a.window = window >= T_total ? 0 : window;
    return a;
}

}  // namespace

extern "C" {

gdr_status gdr_attention_prefill(enum gdr_dtype dt, int B, int T, int T_total, int Hq, int Hkv,
                                 int D, float scale, int window, const void *q, const void *k,
                                 const void *v, const int32_t *cu_seqlens,
                                 const int32_t *cu_seqlens_host, void *o, float *lse,
                                 void *stream) {
    const char *what = "gdr_attention_prefill";
    const gdr_status st = check_prompts(what, dt, B, T, T_total, Hq, Hkv, D, scale, window,
                                        cu_seqlens, cu_seqlens_host);
    if (st != GDR_OK) return st;
    if (B == 0 || T_total == 0) return GDR_OK;
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(v, "v");
    REQUIRE_PTR(o, "o");
    REQUIRE_ALIGNED_OR_NULL(lse, "lse");
    if (cu_seqlens) REQUIRE_I32(cu_seqlens, "cu_seqlens");
    gdr::PromptArgs a = prompt_args(B, T, T_total, Hq, Hkv, scale, window, q, k, v, cu_seqlens);
    a.o = o; a.lse = lse;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_attention_prefill(dt == GDR_BF16, D, a, s), s, what);
}

size_t gdr_attention_backward_workspace_bytes(enum gdr_dtype dt, int B, int T_total, int Hq,
                                              int Hkv, int D) {
    if (B <= 0 || T_total <= 0 ||
        check_prompts("gdr_attention_backward_workspace_bytes", dt, B, 0, T_total, Hq, Hkv, D, 1.f,
                      0, kAnyOffsets, nullptr) != GDR_OK)
        return 0;
    return gdr::attention_backward_workspace(dt == GDR_BF16, B, T_total, Hq, Hkv, D);
}

gdr_status gdr_attention_backward(enum gdr_dtype dt, int B, int T, int T_total, int Hq, int Hkv,
                                  int D, float scale, int window, const void *q, const void *k,
                                  const void *v, const int32_t *cu_seqlens,
                                  const int32_t *cu_seqlens_host, const void *o,
                                  const float *lse, const void *d_o, void *dq, void *dk,
                                  void *dv, void *workspace, size_t ws_bytes, void *stream) {
    const char *what = "gdr_attention_backward";
    gdr_status st = check_prompts(what, dt, B, T, T_total, Hq, Hkv, D, scale, window, cu_seqlens,
                                  cu_seqlens_host);
    if (st != GDR_OK) return st;
    if (B == 0 || T_total == 0) return GDR_OK;
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(v, "v");
    REQUIRE_PTR(o, "o");
    REQUIRE_PTR(lse, "lse");
    REQUIRE_PTR(d_o, "d_o");
    REQUIRE_PTR(dq, "dq");
    REQUIRE_PTR(dk, "dk");
    REQUIRE_PTR(dv, "dv");
    if (cu_seqlens) REQUIRE_I32(cu_seqlens, "cu_seqlens");
    st = check_workspace(what, workspace, ws_bytes,
                         gdr::attention_backward_workspace(dt == GDR_BF16, B, T_total, Hq, Hkv, D));
    if (st != GDR_OK) return st;
    gdr::PromptArgs a = prompt_args(B, T, T_total, Hq, Hkv, scale, window, q, k, v, cu_seqlens);
    a.o = const_cast<void *>(o); a.lse = const_cast<float *>(lse);
    a.d_o = d_o; a.dq = dq; a.dk = dk; a.dv = dv; a.ws = workspace;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_attention_backward(dt == GDR_BF16, D, a, s), s, what);
}

gdr_status gdr_attention_tree(enum gdr_dtype dt, int B, int n_tok, int Hq, int Hkv, int D,
                              float scale, int window, const void *q, const void *k_cache,
                              const void *v_cache, const int32_t *page_table,
                              const int32_t *page_table_host, int max_pages, int page_size,
                              int num_pages, const int32_t *seq_lens, const int32_t *parents,
                              void *o, void *workspace, size_t ws_bytes, void *stream) {
    const char *what = "gdr_attention_tree";
    gdr_status st = check_cache(what, dt, B, Hkv, D, max_pages, page_size, num_pages);
    if (st == GDR_OK) st = check_heads(what, dt, Hq, Hkv, D, scale, window);
    if (st != GDR_OK) return st;
    if (n_tok < 0 || n_tok > kMaxDrafts)
        return fail(n_tok < 0 ? GDR_EINVAL : GDR_EUNSUPPORTED, "%s: n_tok = %d drafts; 0 to %d", what,
                    n_tok, kMaxDrafts);
    if (reaches(B, n_tok, Hq, kMaxQueryRows))
        return fail(GDR_EUNSUPPORTED, "%s: %d x %d x %d query rows exceed %lld", what, B, n_tok, Hq,
                    kMaxQueryRows);
    if (page_table_host) {
        st = check_table(what, "page_table", page_table_host, B, max_pages, num_pages, nullptr);
        if (st != GDR_OK) return st;
    }
    if (B == 0 || n_tok == 0) return GDR_OK;
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(o, "o");
    REQUIRE_I32(seq_lens, "seq_lens");
    REQUIRE_I32(parents, "parents");
    if (max_pages > 0) REQUIRE_I32(page_table, "page_table");
    if (num_pages > 0) {
        REQUIRE_PTR(k_cache, "k_cache");
        REQUIRE_PTR(v_cache, "v_cache");
    }
    st = check_workspace(what, workspace, ws_bytes,
                         gdr_attention_workspace_bytes(B, n_tok, Hq, Hkv, D, max_pages, page_size, 0));
    if (st != GDR_OK) return st;
    gdr::AttnArgs a{};
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    // without pages every token is absent: the kernels see empty sequences
    a.map = gdr::PageMap{page_table, num_pages > 0 ? max_pages : 0, page_shift_of(page_size),
                         num_pages};
    a.seq_lens = seq_lens; a.parents = parents; a.o = o; a.ws = workspace;
    a.B = B; a.n = n_tok; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
    a.scale = scale; a.window = window;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_attention_tree(dt == GDR_BF16, D, a, s), s, what);
}

gdr_status gdr_cache_accept(enum gdr_dtype dt, int B, int n_tok, int Hkv, int D,
                            const int32_t *page_table, int max_pages, int page_size,
                            int num_pages, const int32_t *seq_lens, const int32_t *parents,
                            const int32_t *leaf, void *k_cache, void *v_cache, float *scores,
                            int32_t *new_lens, int32_t *path, void *stream) {
    const char *what = "gdr_cache_accept";
    const gdr_status st = check_cache(what, dt, B, Hkv, D, max_pages, page_size, num_pages);
    if (st != GDR_OK) return st;
    if (n_tok < 0 || n_tok > kMaxDrafts)
        return fail(n_tok < 0 ? GDR_EINVAL : GDR_EUNSUPPORTED, "%s: n_tok = %d drafts; 0 to %d", what,
                    n_tok, kMaxDrafts);
    if ((long long)B * Hkv >= kMaxPairs)
        return fail(GDR_EUNSUPPORTED, "%s: %lld (sequence, head) pairs exceed %lld", what,
                    (long long)B * Hkv, kMaxPairs);
    if (B == 0) return GDR_OK;
    REQUIRE_I32(seq_lens, "seq_lens");
    REQUIRE_I32(leaf, "leaf");
    REQUIRE_I32(new_lens, "new_lens");
    if (n_tok > 0) {
        REQUIRE_I32(parents, "parents");
        REQUIRE_I32(path, "path");
    }
    if (max_pages > 0) REQUIRE_I32(page_table, "page_table");
    if (num_pages > 0) {
        REQUIRE_PTR(k_cache, "k_cache");
        REQUIRE_PTR(v_cache, "v_cache");
    }
    REQUIRE_ALIGNED_OR_NULL(scores, "scores");
    gdr::AcceptArgs a{};
    a.k_cache = k_cache; a.v_cache = v_cache; a.scores = scores;
    a.map = gdr::PageMap{page_table, max_pages, page_shift_of(page_size), num_pages};
    a.seq_lens = seq_lens; a.parents = parents; a.leaf = leaf;
    a.new_lens = new_lens; a.path = path;
    a.B = B; a.n = n_tok; a.Hkv = Hkv;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_cache_accept(D * (dt == GDR_BF16 ? 2 : 4), a, s), s, what);
}

gdr_status gdr_cache_resize(int B, int max_pages, int page_size, int num_pages,
                            int32_t *page_table, const int32_t *seq_lens, const int32_t *want,
                            int32_t *new_lens, int32_t *cu_seqlens, int32_t *free_pages,
                            void *stream) {
    const char *what = "gdr_cache_resize";
    if (B < 0 || max_pages < 0 || page_size < 1 || num_pages < 0)
        return fail(GDR_EINVAL, "%s: bad sizes B=%d max_pages=%d page_size=%d num_pages=%d", what, B,
                    max_pages, page_size, num_pages);
    if (num_pages > gdr::kMaxPages)
        return fail(GDR_EUNSUPPORTED, "%s: %d pages exceed %d", what, num_pages, gdr::kMaxPages);
    if ((long long)max_pages * page_size >= (1LL << 30))
        return fail(GDR_EUNSUPPORTED, "%s: a table of %d pages of %d tokens is too long", what,
                    max_pages, page_size);
    // (sums of lengths are 32-bit numbers)
    if (B >= (1 << 30) || ((long long)num_pages + B) * page_size >= (1LL << 31))
        return fail(GDR_EUNSUPPORTED, "%s: %d pages of %d tokens and %d sequences are too many", what,
                    num_pages, page_size, B);
    if (B > 0) {
        if (max_pages > 0) REQUIRE_I32(page_table, "page_table");
        REQUIRE_I32(seq_lens, "seq_lens");
        REQUIRE_I32(want, "want");
        REQUIRE_I32(new_lens, "new_lens");
    }
    if (cu_seqlens) REQUIRE_I32(cu_seqlens, "cu_seqlens");
    if (free_pages) REQUIRE_I32(free_pages, "free_pages");
    if (B == 0 && !cu_seqlens && !free_pages) return GDR_OK;
    gdr::ResizeArgs a{};
    a.table = page_table; a.seq_lens = seq_lens; a.want = want; a.new_lens = new_lens;
    a.cu_seqlens = cu_seqlens; a.free_pages = free_pages;
    a.B = B; a.max_pages = max_pages; a.page_size = page_size; a.num_pages = num_pages;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdr::launch_cache_resize(a, s), s, what);
}

}  // extern "C"

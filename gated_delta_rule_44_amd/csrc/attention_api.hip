// attention_api.hip -- the C ABI declared in include/gdr_attention.h: host-side
// argument checks and launches on the caller's stream.  Every check runs
// before the first HIP call, so a rejected call has no side effects.  No C++
// exception crosses the interface.
#include <math.h>

#include "../../include/gdr_attention.h"
#include "api_util.h"
#include "prompt_internal.h"

namespace {

using gdr::aligned16;
using gdr::check_workspace;
using gdr::fail;
using gdr::finish;

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

#define REQUIRE_I32(p, name)                                                       \
    do {                                                                           \
        if (!(p)) return fail(GDR_EINVAL, "%s: %s is NULL", what, name);           \
        if (!aligned4(p)) return fail(GDR_EINVAL, "%s: %s is not 4-byte aligned",  \
                                      what, name);                                 \
    } while (0)

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
    // a launch holds fewer than 2^32 threads: 256 for 128 rows of a head, and a
    // sequence may leave one block unused
    if (T_total >= (1 << 30) || B >= (1 << 24) || (long long)T_total * Hq >= (1LL << 31) ||
        ((long long)T_total / 128 + B) * Hq >= (1LL << 24))
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

}  // extern "C"

// cache_check.h -- host-side checks of the paged cache's arguments, shared by
// the C entry points.  Internal to the library.
#pragma once

#include <stdint.h>

#include "api_util.h"

namespace gdr {

// A launch holds fewer than 2^32 threads: rows of new tokens (up to 32
// threads each), query rows (256 threads), trimmed pairs (1,024 threads)
constexpr long long kMaxRows = 1LL << 26, kMaxQueryRows = 1LL << 23, kMaxPairs = 1LL << 21;

// a tree's drafts are bits of a word
constexpr int kMaxDrafts = 64;

inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

#define REQUIRE_I32(p, name)                                                       \
    do {                                                                           \
        if (!(p)) return fail(GDR_EINVAL, "%s: %s is NULL", what, name);           \
        if (!aligned4(p)) return fail(GDR_EINVAL, "%s: %s is not 4-byte aligned",  \
                                      what, name);                                 \
    } while (0)

// a * b * c >= limit, for non-negative factors whose product may not fit
inline bool reaches(long long a, long long b, long long c, long long limit) {
    return (__int128)a * b * c >= limit;
}

// the log2 of a supported page size, or -1
inline int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// dtype, width, heads and the cache's geometry
inline gdr_status check_cache(const char *what, int dt, int B, int Hkv, int D, int max_pages,
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
inline gdr_status check_table(const char *what, const char *name, const int32_t *t, int B,
                              int max_pages, int num_pages, unsigned char *once) {
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

}  // namespace gdr

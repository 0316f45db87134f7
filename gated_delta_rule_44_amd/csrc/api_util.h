// api_util.h -- host-side helpers shared by the C entry points: the error
// text, argument checks, and the end of a call.  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr.h"

namespace gdr {

// sets the thread's error text and returns code
gdr_status fail(gdr_status code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// the status of a call whose launches returned `launch` (GDR_DEBUG: after a
// synchronisation)
gdr_status finish(hipError_t launch, hipStream_t s, const char *what);
gdr_status check_workspace(const char *what, const void *ws, size_t ws_bytes, size_t need);

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace gdr

#define REQUIRE_PTR(p, name)                                                        \
    do {                                                                            \
        if (!(p)) return fail(GDR_EINVAL, "%s: %s is NULL", what, name);            \
        if (!aligned16(p)) return fail(GDR_EINVAL, "%s: %s is not 16-byte aligned", \
                                       what, name);                                 \
    } while (0)
#define REQUIRE_ALIGNED_OR_NULL(p, name)                                            \
    do {                                                                            \
        if ((p) && !aligned16(p)) return fail(GDR_EINVAL,                           \
                                              "%s: %s is not 16-byte aligned",      \
                                              what, name);                          \
    } while (0)

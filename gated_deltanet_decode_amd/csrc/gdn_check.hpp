// gdn_check.hpp - argument checks and error reporting shared by the C-ABI
// sources (gdn_api.cpp, gdn_serve_api.cpp).  All validation happens on the
// host before anything is enqueued.
#pragma once

#include "gdn.h"

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

#include "gdn_launch.hpp"

namespace gdn {

// The thread's error text (gdn_last_error), defined in gdn_api.cpp.
void clear_error();
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// GDN_OK, or GDN_ERR_HIP with `what` and the runtime's message.
int hip_status(hipError_t e, const char *what);

#define GDN_TRY(expr)               \
    do {                            \
        const int rc__ = (expr);    \
        if (rc__ != GDN_OK) return rc__; \
    } while (0)

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Do [a, a+na) and [b, b+nb) share a byte?
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

struct Buf {
    const char *name;
    const void *p;
    size_t bytes;
};

// Every output must be disjoint from every other listed buffer.
inline int check_alias(const Buf *outs, int n_out, const Buf *all, int n_all) {
    for (int i = 0; i < n_out; ++i)
        for (int j = 0; j < n_all; ++j) {
            if (outs[i].p == all[j].p && outs[i].name == all[j].name) continue;  // itself
            if (overlap(outs[i].p, outs[i].bytes, all[j].p, all[j].bytes))
                return fail(GDN_ERR_ALIAS, "%s overlaps %s", outs[i].name, all[j].name);
        }
    return GDN_OK;
}

inline int check_ptrs(const Buf *bufs, int n, uintptr_t align) {
    for (int i = 0; i < n; ++i) {
        if (!bufs[i].p) return fail(GDN_ERR_NULL, "%s is NULL", bufs[i].name);
        if (!aligned(bufs[i].p, align))
            return fail(GDN_ERR_ALIGN, "%s (%p) is not %u-byte aligned", bufs[i].name, bufs[i].p,
                        static_cast<unsigned>(align));
    }
    return GDN_OK;
}

inline int check_dims(const gdn_dims *d) {
    if (!d) return fail(GDN_ERR_NULL, "dims is NULL");
    if (d->n_v_heads < 1 || d->n_k_heads < 1)
        return fail(GDN_ERR_SHAPE, "head counts must be >= 1 (n_v_heads=%d, n_k_heads=%d)",
                    d->n_v_heads, d->n_k_heads);
    if (d->n_v_heads % d->n_k_heads != 0)
        return fail(GDN_ERR_SHAPE, "n_v_heads=%d is not a multiple of n_k_heads=%d",
                    d->n_v_heads, d->n_k_heads);
    if (d->d_k != kHeadDim || d->d_v != kHeadDim)
        return fail(GDN_ERR_SHAPE, "only d_k = d_v = %d is supported (got d_k=%d, d_v=%d)",
                    kHeadDim, d->d_k, d->d_v);
    return GDN_OK;
}

// Heads of one call map to workgroups along grid x, and the persistent
// kernels count 16 row tiles per head in a 32-bit index that may run up to
// one grid stride (at most 65536 tiles) past the last tile.
inline int check_batch(const gdn_dims *d, int64_t B, const char *what) {
    if (B < 1) return fail(GDN_ERR_SHAPE, "%s must be >= 1 (got %lld)", what, (long long)B);
    const int64_t limit = (static_cast<int64_t>(INT32_MAX) - 65536) / 16;   // 134213631
    if (B * d->n_v_heads > limit)
        return fail(GDN_ERR_SHAPE, "B * n_v_heads = %lld exceeds %lld",
                    (long long)(B * d->n_v_heads), (long long)limit);
    return GDN_OK;
}

}  // namespace gdn

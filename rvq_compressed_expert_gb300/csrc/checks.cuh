// Argument checks shared by the C entry points of waste_dense.h and waste_train.h (host side).
#pragma once

#include <cstdarg>
#include <cstdio>

#include "dense.cuh"

namespace wm {
namespace dense {

inline int fail(int code, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return code;
}
inline int ok() {
    set_last_error("");
    return WASTE_OK;
}
inline int done(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return ok();
    cudaGetLastError(); // not left for the next call to find
    return fail(WASTE_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}
constexpr int32_t kMostRows = 1 << 30; // rows and columns of anything: their tiles' indices fit 32 bits
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool half_type(int t) { return t == WASTE_ACT_BF16 || t == WASTE_ACT_F16; }
inline bool any_type(int t) { return t == WASTE_ACT_F32 || half_type(t); }

// NULL or misaligned pointers of a call; names in the order of the pointers.
inline int check_ptrs(const void *const *p, const char *const *name, int n) {
    for (int i = 0; i < n; ++i) {
        if (!p[i]) return fail(WASTE_EINVAL, "%s is NULL", name[i]);
        if (!aligned(p[i], 16)) return fail(WASTE_EINVAL, "%s must be 16-byte aligned", name[i]);
    }
    return WASTE_OK;
}

// Memory of a call: rows of row_bytes, pitch bytes apart.
struct Span {
    const void *p;
    size_t row_bytes;
    const char *name;
    size_t rows = 1, pitch = 0;
};
// Whether a (one row) and b share a byte.
inline bool meet(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.row_bytes || !b.row_bytes || !b.rows) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    if (b.rows == 1) return a0 < b0 + b.row_bytes && b0 < a0 + a.row_bytes;
    // the first row of b that ends behind a's start
    const size_t past = a0 < b0 + b.row_bytes ? 0 : a0 - b0 - b.row_bytes;
    const size_t i = a0 < b0 + b.row_bytes ? 0 : b.pitch ? past / b.pitch + 1 : b.rows;
    return i < b.rows && b0 + i * b.pitch < a0 + a.row_bytes;
}
// Every one of the first n spans, which a call writes, lies apart from all others.
inline int check_apart(const Span *s, int n, int all) {
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < all; ++j)
            if (meet(s[i], s[j])) return fail(WASTE_EINVAL, "%s overlaps %s", s[i].name, s[j].name);
    return WASTE_OK;
}

inline int check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return WASTE_OK;
    if (!ws || !aligned(ws, 256)) return fail(WASTE_EINVAL, "workspace is NULL or not 256-byte aligned");
    if (have < need) return fail(WASTE_EINVAL, "workspace of %zu bytes, %zu needed", have, need);
    return WASTE_OK;
}

} // namespace dense
} // namespace wm

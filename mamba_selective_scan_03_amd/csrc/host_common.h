// host_common.h - what the host entry points of the C ABI share: the calling thread's last HIP
// error, and the checks of addresses, alignment and overlap that run before any launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/jscan.h"

namespace jscan {
namespace host {

// One variable for the whole library, not exported.
extern __thread int g_last_hip_error __attribute__((visibility("hidden")));

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi), empty when lo == hi
};

inline Span span(const void *p, int64_t bytes) {
    Span s;
    if (p && bytes > 0) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + static_cast<uintptr_t>(bytes);
    }
    return s;
}

inline bool overlaps(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// Rows of `width` bytes that start every `ld` bytes: a strided view.
struct Rows {
    const void *p = nullptr;
    int64_t rows = 0, width = 0, ld = 0;
};

inline Span span(const Rows &r) { return span(r.p, r.rows > 0 ? (r.rows - 1) * r.ld + r.width : 0); }

// Whether two strided views share a byte.  Views of one row stride may interleave (the halves of
// one wider buffer); views of different strides are taken to overlap when their extents do.
inline bool overlaps(const Rows &a, const Rows &b) {
    if (!overlaps(span(a), span(b))) return false;
    if (a.ld != b.ld || a.ld <= 0) return true;
    int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % a.ld;
    if (off < 0) off += a.ld;
    return !(off >= a.width && off + b.width <= a.ld);
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

inline int64_t elem_bytes(jscan_dtype dt) { return dt == JSCAN_BF16 ? 2 : 4; }

inline jscan_status launch_status() {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        g_last_hip_error = static_cast<int>(e);
        return JSCAN_ERR_HIP;
    }
    return JSCAN_OK;
}

// Largest grid the launchers accept (work-group counts and row indices are 32-bit ints).
constexpr int64_t kMaxBlocks = (int64_t)1 << 30;

// Work-items that one dimension of a launch can count.
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;

// Sizes of padded batches that the index arithmetic of the kernels holds: rows of D and grids in 32 bits, byte
// offsets in 63.
inline bool shape_ok(int64_t batch, int64_t L, int64_t D) {
    return batch >= 0 && L >= 0 && D >= 0 && D <= (1 << 24) && batch <= (1 << 20) && L < ((int64_t)1 << 31) &&
           batch * ((D + 63) / 64) <= kMaxBlocks;
}
inline bool ld_ok(int64_t ld, int64_t rows, int64_t D) { return ld >= D && (rows == 0 || ld <= ((int64_t)1 << 58) / rows); }

struct Pair {
    const void *p;
    int64_t ld;
};

inline Rows rows_of(Pair t, int64_t rows, int64_t D, int64_t es) { return Rows{t.p, t.p ? rows : 0, D * es, t.ld * es}; }
inline Rows flat(const void *p, int64_t bytes) { return Rows{p, p && bytes > 0 ? 1 : 0, bytes, bytes}; }

// Whether an output shares memory with an input or with another output.
template <int NO, int NI> bool any_overlap(const Rows (&out)[NO], const Rows (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(out[i], in[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlaps(out[i], out[j])) return true;
    }
    return false;
}

}  // namespace host
}  // namespace jscan

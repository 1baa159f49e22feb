// token_rows.h - strided [batch][L][D] tensors and padded sequences, as the kernels over whole sequences take them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace jscan {

// A [batch][L][D] tensor whose token rows start every ld elements (batch stride L * ld).
template <typename T> struct TokenRows {
    T *p;
    int64_t ld;
};

// Tokens of sequence b that count: lengths[b] clamped to [0, L], or L without lengths.
__device__ __forceinline__ int64_t tokens_of(const int32_t *lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > L ? L : n);
}

}  // namespace jscan

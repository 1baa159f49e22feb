// int8_kernels.h - a linear layer in 8-bit integers: activations quantised row by row (token by
// token), weights held as int8 with a scale for each output channel, products summed in int32.
//
//     s[m] = max(max_k |x[m][k]| / 127, 2^-126),   q[m][k] = rint(x[m][k] * (1 / s[m]))
//     out[m][n] = (sum_k q[m][k] w[n][k]) * s[m] * s_w[n] + bias[n]
//
// The sum is exact (K <= 131056 keeps 128 * 128 * K below 2^31); it is rounded to fp32 once, and the
// scales and the bias are applied in fp32 before the one rounding to the output type.
#pragma once

#include "mfma_common.h"

namespace jscan {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// 16x16 tile of int32 sums, 64 deep.  Both operands take 16 consecutive bytes of k per lane, at
// k = 16 * (l / 16), from row (column) l % 16; lane l holds result rows 4 * (l / 16) + i of column l % 16.
__device__ __forceinline__ i32x4_t mfma_i8(i32x4_t a, i32x4_t b, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

namespace quant {
constexpr int kThreads = 256;
}

// The scale of a row whose largest magnitude is amax.  The lower bound keeps 1 / s finite; a row of
// zeros takes it and quantises to zeros.
__device__ __forceinline__ float row_scale(float amax) { return fmaxf(amax / 127.0f, 0x1.0p-126f); }

// One work-group per row, which is read twice (the second time from the caches).
template <typename E>
__global__ __launch_bounds__(quant::kThreads) void quantize_rows_kernel(const typename E::store_t *__restrict__ x,
                                                                        int8_t *__restrict__ q,
                                                                        float *__restrict__ scale, int64_t K,
                                                                        int64_t ld_x) {
    __shared__ float part[quant::kThreads / 64];
    const int64_t m = blockIdx.x;
    const typename E::store_t *row = x + m * ld_x;
    // a NaN or an infinity anywhere in the row makes its sum with zero weights NaN
    float amax = 0.0f, poison = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += quant::kThreads) {
        const float v = E::load(row + k);
        amax = fmaxf(amax, fabsf(v));
        poison = __builtin_fmaf(v, 0.0f, poison);
    }
    amax = poison == 0.0f ? amax : __builtin_inff();
    for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const bool finite = amax < __builtin_inff();
    const float s = finite ? row_scale(amax) : __builtin_nanf("");
    const float r = 1.0f / s;
    for (int64_t k = threadIdx.x; k < K; k += quant::kThreads)
        q[m * K + k] = finite ? (int8_t)__builtin_rintf(E::load(row + k) * r) : (int8_t)0;
    if (threadIdx.x == 0) scale[m] = s;
}

// One wave per 16 x 16 tile of the output, operands straight from memory.
template <typename E>
__global__ __launch_bounds__(64) void matmul_i8_kernel(const int8_t *__restrict__ q, const float *__restrict__ sq,
                                                       const int8_t *__restrict__ w, const float *__restrict__ sw,
                                                       const float *__restrict__ bias,
                                                       typename E::store_t *__restrict__ out, int64_t M, int64_t N,
                                                       int64_t K, int64_t ld_out, int n_tiles) {
    const int64_t m0 = (int64_t)(blockIdx.x / n_tiles) * 16, n0 = (int64_t)(blockIdx.x % n_tiles) * 16;
    const int l = threadIdx.x, r16 = l & 15, g4 = l >> 4;
    const int8_t *qr = q + min(m0 + r16, M - 1) * K, *wr = w + min(n0 + r16, N - 1) * K;
    i32x4_t acc = {0, 0, 0, 0};
    for (int64_t k = 16 * g4; k - 16 * g4 < K; k += 64) {
        i32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (k < K) {   // K is a multiple of 16
            a = *reinterpret_cast<const i32x4_t *>(qr + k);
            b = *reinterpret_cast<const i32x4_t *>(wr + k);
        }
        acc = mfma_i8(a, b, acc);
    }
    const int64_t n = n0 + r16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * g4 + i;
        if (m < M && n < N) {
            const float v = (float)acc[i] * sq[m] * sw[n];
            E::store(out + m * ld_out + n, bias ? v + bias[n] : v);
        }
    }
}

}  // namespace jscan

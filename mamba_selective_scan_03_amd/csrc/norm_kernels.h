// norm_kernels.h - root-mean-square norm with the residual's addition in front of it, its output in the tensor's type or
// in 8 bits with a scale for each row, and its backward pass.
//
//     t = x + residual, rounded to the type (the residual stream as it is kept);   r = 1 / sqrt(mean_k t^2 + eps)
//     y = (t gain) r;   in 8 bits  s = max(max_k |y| (1 / 127), 2^-126),  q = rint(y (1 / s))
//     backward, with g = dy gain:   dt = r (g - t r mean_k(g t r)) + dtotal,   dgain = sum over rows of dy t r
//
// Memory bounds them (bf16: 8, 7 and 8 bytes an element for about 15 instructions): a row stays in the registers of
// one work-group between its sums and its outputs, so every byte moves once; work-groups go on to further rows
// and have the next one on its way while they finish one, the gain (and its gradient) in registers.
#pragma once

#include <type_traits>

#include "int8_kernels.h"

namespace jscan {

// M rows of K values, ld elements apart.
template <typename T> struct NormRows {
    T *p;
    int64_t ld;
};

namespace norm {

// 16 bytes of a row, aligned to the element alone: any row stride takes the same loads.
template <typename E> struct Piece;
template <> struct Piece<BF16> {
    static constexpr int n = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    static __device__ __forceinline__ uint32_t mask(int lo, int i) {   // word i without the elements below lo
        return lo <= 2 * i ? ~0u : lo == 2 * i + 1 ? 0xffff0000u : 0u;
    }
    static __device__ __forceinline__ void unpack(raw w, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[8]) {
        return raw{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
    }
};
template <> struct Piece<F32> {
    static constexpr int n = 4;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
    static __device__ __forceinline__ uint32_t mask(int lo, int i) { return lo <= i ? ~0u : 0u; }
    static __device__ __forceinline__ void unpack(raw w, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[4]) {
        return raw{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};
template <typename E> using Raw = typename Piece<E>::raw;

template <typename E> __device__ __forceinline__ Raw<E> load(const typename E::store_t *p) {
    return *reinterpret_cast<const Raw<E> *>(p);
}
template <typename E> __device__ __forceinline__ void store(typename E::store_t *p, Raw<E> v) {
    *reinterpret_cast<Raw<E> *>(p) = v;
}

// Which kChunks pieces of a row a thread of kWaves waves has: piece j kWaves 64 + thread.  Where the pieces do not divide the
// row the last one reaches back over the one before it: both compute the same outputs, and the sums leave the
// repeated elements out (`keep`, which also empties threads behind the row).  Only the last of a thread's
// pieces can be such a one (the host picks kChunks so).
template <typename E, int kWaves, int kChunks> struct Place {
    static constexpr int n = Piece<E>::n, kThreads = kWaves * 64;
    int at[kChunks];   // first element
    int lo;            // first element of the last piece that counts
    Raw<E> keep;       // as a mask
    __device__ __forceinline__ explicit Place(int K) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) at[j] = min((j * kThreads + (int)threadIdx.x) * n, K - n);
        const int first = ((kChunks - 1) * kThreads + (int)threadIdx.x) * n;
        lo = first < K ? first - at[kChunks - 1] : n;
#pragma unroll
        for (int i = 0; i < 4; ++i) keep[i] = Piece<E>::mask(lo, i);
    }
    __device__ __forceinline__ Raw<E> counted(Raw<E> w, int j) const { return j == kChunks - 1 ? w & keep : w; }
    __device__ __forceinline__ bool live() const { return lo < n; }
};

// Sum of a and, by kMax, maximum or sum of b over a work-group; `part` holds kWaves pairs, of another parity for every
// second call, so that one barrier a call is enough.
template <int kWaves, bool kMax> __device__ __forceinline__ void group_reduce(float &a, float &b, float2 *part) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        a += __shfl_xor(a, o);
        const float other = __shfl_xor(b, o);
        b = kMax ? fmaxf(b, other) : b + other;
    }
    if constexpr (kWaves > 1) {
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = make_float2(a, b);
        __syncthreads();
        a = part[0].x, b = part[0].y;
#pragma unroll
        for (int i = 1; i < kWaves; ++i) {
            a += part[i].x;
            b = kMax ? fmaxf(b, part[i].y) : b + part[i].y;
        }
    }
}

__device__ __forceinline__ float rms_scale(float sum, int K, float eps) {
    return __builtin_amdgcn_rsqf(sum / (float)K + eps);
}

template <typename E, int kChunks> __device__ __forceinline__ void load_gain(float (&g)[kChunks][Piece<E>::n], const float *gain,
                                                                             const int (&at)[kChunks]) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < Piece<E>::n; ++i) g[j][i] = gain[at[j] + i];
}

}  // namespace norm

// Where the norm's output goes: rows of the tensor's type, or int8 rows and their scales.
template <typename E> struct NormOut {
    NormRows<typename E::store_t> y;
    int8_t *q;
    float *scale;
};

// total may be x or residual itself: a row is stored after the work-group's last load of it.
template <typename E, int kWaves, int kChunks, bool kInt8, bool kResidual>
__global__ __launch_bounds__(kWaves * 64) void rms_norm_kernel(NormRows<const typename E::store_t> x,
                                                               NormRows<const typename E::store_t> residual,
                                                               const float *__restrict__ gain, NormOut<E> out,
                                                               NormRows<typename E::store_t> total, int64_t M, int K,
                                                               float eps) {
    using P = norm::Piece<E>;
    using raw = norm::Raw<E>;
    constexpr int n = P::n;
    __shared__ float2 part[2][kWaves];
    const norm::Place<E, kWaves, kChunks> at(K);
    raw xn[kChunks], rn[kChunks];
    auto fetch = [&](int64_t m) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            xn[j] = norm::load<E>(x.p + m * x.ld + at.at[j]);
            if constexpr (kResidual) rn[j] = norm::load<E>(residual.p + m * residual.ld + at.at[j]);
        }
    };
    int64_t m = blockIdx.x;
    fetch(m);
    float g[kChunks][n];
    norm::load_gain<E, kChunks>(g, gain, at.at);
    for (int parity = 0; m < M; m += gridDim.x, parity ^= 1) {
        raw t[kChunks];
        float sum = 0.0f, amax = 0.0f, poison = 0.0f;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            if constexpr (kResidual) {
                float a[n], b[n];
                P::unpack(xn[j], a);
                P::unpack(rn[j], b);
#pragma unroll
                for (int i = 0; i < n; ++i) a[i] += b[i];
                t[j] = P::pack(a);
            } else {
                t[j] = xn[j];
            }
            float f[n];
            P::unpack(at.counted(t[j], j), f);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                sum = __builtin_fmaf(f[i], f[i], sum);
                if constexpr (kInt8) {
                    const float v = f[i] * g[j][i];
                    amax = fmaxf(amax, fabsf(v));
                    poison = __builtin_fmaf(v, 0.0f, poison);
                }
            }
        }
        if (m + gridDim.x < M) fetch(m + gridDim.x);
        if constexpr (kInt8) amax = poison == 0.0f ? amax : __builtin_inff();
        norm::group_reduce<kWaves, true>(sum, amax, part[parity]);
        const float r = norm::rms_scale(sum, K, eps);
        float s = 0.0f, inv = 0.0f;
        bool finite = true;
        if constexpr (kInt8) {
            // (t gain) r rounds in order, so the row's largest |y| is that of its largest |t gain|
            finite = sum < __builtin_inff() && amax * r < __builtin_inff();
            s = finite ? quant::row_scale(amax * r) : __builtin_nanf("");
            inv = 1.0f / s;
            if (threadIdx.x == 0) out.scale[m] = s;
        }
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            if (j == kChunks - 1 && !at.live()) break;
            float f[n];
            P::unpack(t[j], f);
#pragma unroll
            for (int i = 0; i < n; ++i) f[i] = f[i] * g[j][i] * r;
            if constexpr (kInt8) {
                uint32_t *dst = reinterpret_cast<uint32_t *>(out.q + m * K + at.at[j]);
#pragma unroll
                for (int i = 0; i < n / 4; ++i) dst[i] = finite ? quant::pack4(f + 4 * i, inv) : 0u;
            } else {
                norm::store<E>(out.y.p + m * out.y.ld + at.at[j], P::pack(f));
            }
            if (kResidual && total.p) norm::store<E>(total.p + m * total.ld + at.at[j], t[j]);
        }
    }
}

// Rows shorter than a piece or longer than the registers hold: one element a thread at a time, read again for the
// outputs (from the stored total where there is one, by the thread that stored it).
template <typename E, int kWaves, bool kInt8>
__global__ __launch_bounds__(kWaves * 64) void rms_norm_any_kernel(NormRows<const typename E::store_t> x,
                                                                   NormRows<const typename E::store_t> residual,
                                                                   const float *__restrict__ gain, NormOut<E> out,
                                                                   NormRows<typename E::store_t> total, int64_t M, int K,
                                                                   float eps) {
    __shared__ float2 part[2][kWaves];
    int parity = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, parity ^= 1) {
        const typename E::store_t *xr = x.p + m * x.ld;
        auto value = [&](int k) {
            float v = E::load(xr + k);
            if (residual.p) {
                typename E::store_t rounded;
                E::store(&rounded, v + E::load(residual.p + m * residual.ld + k));
                v = E::load(&rounded);
            }
            return v;
        };
        const bool kept = residual.p && total.p;
        float sum = 0.0f, amax = 0.0f, poison = 0.0f;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float t = value(k), v = t * gain[k];
            if (kept) E::store(total.p + m * total.ld + k, t);
            sum = __builtin_fmaf(t, t, sum);
            amax = fmaxf(amax, fabsf(v));
            poison = __builtin_fmaf(v, 0.0f, poison);
        }
        amax = poison == 0.0f ? amax : __builtin_inff();
        norm::group_reduce<kWaves, true>(sum, amax, part[parity]);
        const float r = norm::rms_scale(sum, K, eps);
        const bool finite = sum < __builtin_inff() && amax * r < __builtin_inff();
        const float s = finite ? quant::row_scale(amax * r) : __builtin_nanf(""), inv = 1.0f / s;
        if (kInt8 && threadIdx.x == 0) out.scale[m] = s;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float t = kept ? E::load(total.p + m * total.ld + k) : value(k), y = t * gain[k] * r;
            if constexpr (kInt8) out.q[m * K + k] = finite ? (int8_t)__builtin_rintf(y * inv) : (int8_t)0;
            else E::store(out.y.p + m * out.y.ld + k, y);
        }
    }
}

// The backward pass; dx may be dtotal itself.  partial[work-group][K]: the gain's gradient of a work-group's rows.
template <typename E, int kWaves, int kChunks, bool kAdd>
__global__ __launch_bounds__(kWaves * 64) void rms_norm_backward_kernel(
    NormRows<const typename E::store_t> total, const float *__restrict__ gain, NormRows<const typename E::store_t> dy,
    NormRows<const typename E::store_t> dtotal, NormRows<typename E::store_t> dx, float *__restrict__ partial, int64_t M,
    int K, float eps) {
    using P = norm::Piece<E>;
    using raw = norm::Raw<E>;
    constexpr int n = P::n;
    __shared__ float2 part[2][kWaves];
    const norm::Place<E, kWaves, kChunks> at(K);
    raw tn[kChunks], yn[kChunks], an[kChunks];
    auto fetch = [&](int64_t m) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            tn[j] = norm::load<E>(total.p + m * total.ld + at.at[j]);
            yn[j] = norm::load<E>(dy.p + m * dy.ld + at.at[j]);
            if constexpr (kAdd) an[j] = norm::load<E>(dtotal.p + m * dtotal.ld + at.at[j]);
        }
    };
    int64_t m = blockIdx.x;
    fetch(m);
    float g[kChunks][n], dg[kChunks][n];
    norm::load_gain<E, kChunks>(g, gain, at.at);
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < n; ++i) dg[j][i] = 0.0f;
    for (int parity = 0; m < M; m += gridDim.x, parity ^= 1) {
        raw t[kChunks], d[kChunks], a[kChunks];
        float sum = 0.0f, along = 0.0f;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            t[j] = tn[j], d[j] = yn[j];
            if constexpr (kAdd) a[j] = an[j];
            float f[n], e[n];
            P::unpack(at.counted(t[j], j), f);
            P::unpack(at.counted(d[j], j), e);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                sum = __builtin_fmaf(f[i], f[i], sum);
                along = __builtin_fmaf(e[i] * g[j][i], f[i], along);
            }
        }
        if (m + gridDim.x < M) fetch(m + gridDim.x);
        norm::group_reduce<kWaves, false>(sum, along, part[parity]);
        const float r = norm::rms_scale(sum, K, eps), c = along / (float)K * r;   // mean of g t r
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            if (j == kChunks - 1 && !at.live()) break;
            float f[n], e[n], o[n];
            P::unpack(t[j], f);
            P::unpack(d[j], e);
            if constexpr (kAdd) P::unpack(a[j], o);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float t_r = f[i] * r, v = r * __builtin_fmaf(-t_r, c, e[i] * g[j][i]);
                o[i] = kAdd ? v + o[i] : v;
                dg[j][i] = __builtin_fmaf(e[i], t_r, dg[j][i]);
            }
            norm::store<E>(dx.p + m * dx.ld + at.at[j], P::pack(o));
        }
    }
    float *to = partial + (int64_t)blockIdx.x * K;
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (j < kChunks - 1 || i >= at.lo) to[at.at[j] + i] = dg[j][i];
}

// Any other row, as above; a work-group's own row of partial is where it sums the gain's gradient.
template <typename E, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void rms_norm_backward_any_kernel(
    NormRows<const typename E::store_t> total, const float *__restrict__ gain, NormRows<const typename E::store_t> dy,
    NormRows<const typename E::store_t> dtotal, NormRows<typename E::store_t> dx, float *__restrict__ partial, int64_t M,
    int K, float eps) {
    __shared__ float2 part[2][kWaves];
    float *to = partial + (int64_t)blockIdx.x * K;
    for (int k = threadIdx.x; k < K; k += kWaves * 64) to[k] = 0.0f;
    int parity = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, parity ^= 1) {
        const typename E::store_t *t = total.p + m * total.ld, *d = dy.p + m * dy.ld;
        float sum = 0.0f, along = 0.0f;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float f = E::load(t + k);
            sum = __builtin_fmaf(f, f, sum);
            along = __builtin_fmaf(E::load(d + k) * gain[k], f, along);
        }
        norm::group_reduce<kWaves, false>(sum, along, part[parity]);
        const float r = norm::rms_scale(sum, K, eps), c = along / (float)K * r;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float t_r = E::load(t + k) * r, e = E::load(d + k);
            float v = r * __builtin_fmaf(-t_r, c, e * gain[k]);
            if (dtotal.p) v += E::load(dtotal.p + m * dtotal.ld + k);
            E::store(dx.p + m * dx.ld + k, v);
            to[k] = __builtin_fmaf(e, t_r, to[k]);
        }
    }
}

// The sum of the work-groups' rows, 64 columns a work-group: four waves take every fourth row each.
static __global__ __launch_bounds__(256) void norm_gain_kernel(const float *__restrict__ partial, float *__restrict__ dgain,
                                                               int64_t rows, int K) {
    __shared__ float part[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int64_t p = wave; p < rows; p += 4) s += partial[p * K + k];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && k < K) dgain[k] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

}  // namespace jscan

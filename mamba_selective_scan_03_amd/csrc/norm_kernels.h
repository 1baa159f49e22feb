// norm_kernels.h - root-mean-square norm with the residual's addition in front of it, its output in the tensor's type or
// in 8 bits with a scale for each row, and its backward pass.
//
//     t = x + residual, rounded to the type (the residual stream as it is kept);   r = 1 / sqrt(mean_k t^2 + eps)
//     y = (t gain) r;   in 8 bits  s = max(max_k |y| (1 / 127), 2^-126),  q = rint(y (1 / s))
//     backward, with g = dy gain:   dt = r (g - t r mean_k(g t r)) + dtotal,   dgain = sum over rows of dy t r
//
// Memory bounds them (bf16: 8, 7 and 8 bytes an element for about 15 instructions): up to 4096 pieces of 16 bytes a row
// stays in the registers of one work-group between its sums and its outputs, so every byte moves once.  Forward a
// work-group takes one row (more only beyond 2^20 rows).  Backward it goes on to further rows, with the gain and its
// gradient in registers and, with one or four waves, the next rows on their way while it finishes some; with sixteen the
// registers hold one row and none ahead, and the longest rows are read again (kAgain).  Rows shorter than a piece and
// longer ones go element by element and are read twice.
// Measured (bf16 with a residual; us, bytes that cross HBM over time): 16384 x 4096 forward 92, 5.8 TB/s, backward 90 + 5
// for the gain's sum, 6.1; 65536 x 4096 into 8 bits 309, 6.1; one row of 4096 2.4.
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
        return raw{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
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

// kNt: with the non-temporal hint, for tensors that go by.
template <typename E, bool kNt> __device__ __forceinline__ Raw<E> load(const typename E::store_t *p) {
    if constexpr (kNt) return __builtin_nontemporal_load(reinterpret_cast<const Raw<E> *>(p));
    return *reinterpret_cast<const Raw<E> *>(p);
}
template <typename E, bool kNt> __device__ __forceinline__ void store(typename E::store_t *p, Raw<E> v) {
    if constexpr (kNt) __builtin_nontemporal_store(v, reinterpret_cast<Raw<E> *>(p));
    else *reinterpret_cast<Raw<E> *>(p) = v;
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

// A value of another lane: DPP inside rows of 16 lanes (quads by quad_perm, the other quad, the other half by mirrors),
// permlane swaps across them.
template <int kControl> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), kControl, 0xF, 0xF, true));
}
typedef unsigned u32_pair __attribute__((ext_vector_type(2)));
// Every lane's v joined with the other rows': the two results of a swap of v with itself are v and its partner.
template <bool kMax> __device__ __forceinline__ float join(float a, float b) { return kMax ? fmaxf(a, b) : a + b; }
template <bool kMax> __device__ __forceinline__ float wave_reduce(float v) {
    v = join<kMax>(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
    v = join<kMax>(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
    v = join<kMax>(v, dpp<0x141>(v));   // row_half_mirror
    v = join<kMax>(v, dpp<0x140>(v));   // row_mirror
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto across16 = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = join<kMax>(__builtin_bit_cast(float, (unsigned)across16[0]), __builtin_bit_cast(float, (unsigned)across16[1]));
    const unsigned w = __builtin_bit_cast(unsigned, v);
    const auto across32 = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return join<kMax>(__builtin_bit_cast(float, (unsigned)across32[0]), __builtin_bit_cast(float, (unsigned)across32[1]));
}

// Sums of a and, by kMax, maxima or sums of b over a work-group, for kRows rows at once; `part` holds their pairs of
// every wave, another one for every second call, so that one barrier a call is enough.
template <int kWaves, bool kMax, int kRows>
__device__ __forceinline__ void group_reduce(float (&a)[kRows], float (&b)[kRows], float2 (&part)[kRows][kWaves]) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        a[r] = wave_reduce<false>(a[r]);
        b[r] = wave_reduce<kMax>(b[r]);
    }
    if constexpr (kWaves > 1) {
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) part[r][threadIdx.x / 64] = make_float2(a[r], b[r]);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            a[r] = part[r][0].x, b[r] = part[r][0].y;
#pragma unroll
            for (int i = 1; i < kWaves; ++i) a[r] += part[r][i].x, b[r] = join<kMax>(b[r], part[r][i].y);
        }
    }
}

// Rows that a work-group of the backward pass takes at a time: two where a thread has up to two pieces of each (us, one,
// two and four: 65536 x 256 bf16 45, 39, 43; 65536 x 4096 384, 359).  Sixteen waves leave 128 registers a thread,
// which hold one row and none on its way (20000 x 8192 fp32 468 us, with two rows 1922).
constexpr int rows_at_once(int waves, int chunks) { return waves < 16 && chunks <= 2 ? 2 : 1; }
constexpr bool fetches_ahead(int waves) { return waves < 16; }

// 1 / sqrt(mean + eps).  Outside the normal numbers there is none that fp32 squares could give (they have overflowed or
// lost their bits, or the row holds an infinity): NaN, so that every form of the call says so.
__device__ __forceinline__ float rms_scale(float sum, int K, float eps) {
    const float v = sum / (float)K + eps;
    return v >= 0x1.0p-126f && v < __builtin_inff() ? __builtin_amdgcn_rsqf(v) : __builtin_nanf("");
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
template <typename E, int kWaves, int kChunks, bool kInt8, bool kResidual, bool kNt>
__global__ __launch_bounds__(kWaves * 64) void rms_norm_kernel(NormRows<const typename E::store_t> x,
                                                               NormRows<const typename E::store_t> residual,
                                                               const float *__restrict__ gain, NormOut<E> out,
                                                               NormRows<typename E::store_t> total, int64_t M, int K,
                                                               float eps) {
    using P = norm::Piece<E>;
    using raw = norm::Raw<E>;
    constexpr int n = P::n;
    __shared__ float2 part[2][1][kWaves];
    const norm::Place<E, kWaves, kChunks> at(K);
    float g[kChunks][n];
    int parity = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, parity ^= 1) {
        raw t[kChunks], rest[kChunks];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            t[j] = norm::load<E, kNt>(x.p + m * x.ld + at.at[j]);
            if constexpr (kResidual) rest[j] = norm::load<E, kNt>(residual.p + m * residual.ld + at.at[j]);
        }
        if (m == blockIdx.x) norm::load_gain<E, kChunks>(g, gain, at.at);
        float sum[1] = {0.0f}, amax[1] = {0.0f}, poison = 0.0f;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            if constexpr (kResidual) {
                float a[n], b[n];
                P::unpack(t[j], a);
                P::unpack(rest[j], b);
#pragma unroll
                for (int i = 0; i < n; ++i) a[i] += b[i];
                t[j] = P::pack(a);
            }
            float f[n];
            P::unpack(at.counted(t[j], j), f);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                sum[0] = __builtin_fmaf(f[i], f[i], sum[0]);
                if constexpr (kInt8) {
                    const float v = f[i] * g[j][i];
                    amax[0] = fmaxf(amax[0], fabsf(v));
                    poison = __builtin_fmaf(v, 0.0f, poison);
                }
            }
        }
        if constexpr (kInt8) amax[0] = poison == 0.0f ? amax[0] : __builtin_inff();
        norm::group_reduce<kWaves, true, 1>(sum, amax, part[parity]);
        const float r = norm::rms_scale(sum[0], K, eps);
        float inv = 0.0f;
        bool finite = true;
        if constexpr (kInt8) {
            // (t gain) r rounds in order, so the row's largest |y| is that of its largest |t gain|
            finite = sum[0] < __builtin_inff() && amax[0] * r < __builtin_inff();
            const float s = finite ? quant::row_scale(amax[0] * r) : __builtin_nanf("");
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
                norm::store<E, kNt>(out.y.p + m * out.y.ld + at.at[j], P::pack(f));
            }
            if (kResidual && total.p) norm::store<E, kNt>(total.p + m * total.ld + at.at[j], t[j]);
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
    __shared__ float2 part[2][1][kWaves];
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
        float sum[1] = {0.0f}, amax[1] = {0.0f}, poison = 0.0f;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float t = value(k), v = t * gain[k];
            if (kept) E::store(total.p + m * total.ld + k, t);
            sum[0] = __builtin_fmaf(t, t, sum[0]);
            amax[0] = fmaxf(amax[0], fabsf(v));
            poison = __builtin_fmaf(v, 0.0f, poison);
        }
        amax[0] = poison == 0.0f ? amax[0] : __builtin_inff();
        norm::group_reduce<kWaves, true, 1>(sum, amax, part[parity]);
        const float r = norm::rms_scale(sum[0], K, eps);
        const bool finite = sum[0] < __builtin_inff() && amax[0] * r < __builtin_inff();
        const float s = finite ? quant::row_scale(amax[0] * r) : __builtin_nanf(""), inv = 1.0f / s;
        if (kInt8 && threadIdx.x == 0) out.scale[m] = s;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float t = kept ? E::load(total.p + m * total.ld + k) : value(k), y = t * gain[k] * r;
            if constexpr (kInt8) out.q[m * K + k] = finite ? (int8_t)__builtin_rintf(y * inv) : (int8_t)0;
            else E::store(out.y.p + m * out.y.ld + k, y);
        }
    }
}

// The backward pass; dx may be dtotal itself.  A work-group takes kRows rows at a time, the next ones on their way (kAhead); rows
// behind the last one read it again and count nothing.  partial[work-group][K]: the gain's gradient of a
// work-group's rows.
template <typename E, int kWaves, int kChunks, bool kAdd, bool kNt>
__global__ __launch_bounds__(kWaves * 64) void rms_norm_backward_kernel(
    NormRows<const typename E::store_t> total, const float *__restrict__ gain, NormRows<const typename E::store_t> dy,
    NormRows<const typename E::store_t> dtotal, NormRows<typename E::store_t> dx, float *__restrict__ partial, int64_t M,
    int K, float eps) {
    using P = norm::Piece<E>;
    using raw = norm::Raw<E>;
    constexpr int n = P::n, kRows = norm::rows_at_once(kWaves, kChunks);
    constexpr bool kAhead = norm::fetches_ahead(kWaves);
    // the longest rows are read again for their gradients, from the caches: 128 registers do not hold them beside
    // the gain and its gradient (us, and where they are held and spill: 8000 x 30000 bf16 740, 857; 8000 x 20000 257, 307).
    // Four pieces of bf16 spill even so, about 60 registers of gain and gradient; three up to 4
    constexpr bool kAgain = kWaves == 16 && kChunks * n > 16;
    __shared__ float2 part[2][kRows][kWaves];
    const norm::Place<E, kWaves, kChunks> at(K);
    raw tn[kRows][kChunks], yn[kRows][kChunks], an[kRows][kChunks];
    auto fetch = [&](int64_t m0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t m = min(m0 + r, M - 1);
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                tn[r][j] = norm::load<E, kNt && !kAgain>(total.p + m * total.ld + at.at[j]);
                yn[r][j] = norm::load<E, kNt && !kAgain>(dy.p + m * dy.ld + at.at[j]);
                if constexpr (kAdd && !kAgain) an[r][j] = norm::load<E, kNt>(dtotal.p + m * dtotal.ld + at.at[j]);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t m0 = (int64_t)blockIdx.x * kRows;
    if constexpr (kAhead) fetch(m0);
    float g[kChunks][n], dg[kChunks][n];
    norm::load_gain<E, kChunks>(g, gain, at.at);
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < n; ++i) dg[j][i] = 0.0f;
    for (int parity = 0; m0 < M; m0 += step, parity ^= 1) {
        raw t[kRows][kChunks], d[kRows][kChunks], a[kRows][kChunks];
        float sum[kRows], along[kRows];
        if constexpr (!kAhead) fetch(m0);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            sum[r] = along[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                t[r][j] = tn[r][j], d[r][j] = yn[r][j];
                if constexpr (kAdd && !kAgain) a[r][j] = an[r][j];
                float f[n], e[n];
                P::unpack(at.counted(t[r][j], j), f);
                P::unpack(at.counted(d[r][j], j), e);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    sum[r] = __builtin_fmaf(f[i], f[i], sum[r]);
                    along[r] = __builtin_fmaf(e[i] * g[j][i], f[i], along[r]);
                }
            }
        }
        if (kAhead && m0 + step < M) fetch(m0 + step);
        norm::group_reduce<kWaves, false, kRows>(sum, along, part[parity]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t m = m0 + r;
            if (m >= M) break;
            const float rms = norm::rms_scale(sum[r], K, eps), c = along[r] / (float)K * rms;   // mean of g t rms
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                if (j == kChunks - 1 && !at.live()) break;
                if constexpr (kAgain) {
                    t[r][j] = norm::load<E, false>(total.p + m * total.ld + at.at[j]);
                    d[r][j] = norm::load<E, false>(dy.p + m * dy.ld + at.at[j]);
                    if constexpr (kAdd) a[r][j] = norm::load<E, false>(dtotal.p + m * dtotal.ld + at.at[j]);
                }
                float f[n], e[n], o[n];
                P::unpack(t[r][j], f);
                P::unpack(d[r][j], e);
                if constexpr (kAdd) P::unpack(a[r][j], o);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float t_r = f[i] * rms, v = rms * __builtin_fmaf(-t_r, c, e[i] * g[j][i]);
                    o[i] = kAdd ? v + o[i] : v;
                    dg[j][i] = __builtin_fmaf(e[i], t_r, dg[j][i]);
                }
                typename E::store_t *to = dx.p + m * dx.ld + at.at[j];
                if (kAgain && j == kChunks - 1 && at.lo > 0) {
                    // where dx is dtotal and rows are read again, the repeated elements may hold their gradient
                    // already: only the thread that counts an element writes it
#pragma unroll
                    for (int i = 0; i < n; ++i)
                        if (i >= at.lo) E::store(to + i, o[i]);
                } else {
                    norm::store<E, kNt>(to, P::pack(o));
                }
            }
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
    __shared__ float2 part[2][1][kWaves];
    float *to = partial + (int64_t)blockIdx.x * K;
    for (int k = threadIdx.x; k < K; k += kWaves * 64) to[k] = 0.0f;
    int parity = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, parity ^= 1) {
        const typename E::store_t *t = total.p + m * total.ld, *d = dy.p + m * dy.ld;
        float sum[1] = {0.0f}, along[1] = {0.0f};
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float f = E::load(t + k);
            sum[0] = __builtin_fmaf(f, f, sum[0]);
            along[0] = __builtin_fmaf(E::load(d + k) * gain[k], f, along[0]);
        }
        norm::group_reduce<kWaves, false, 1>(sum, along, part[parity]);
        const float r = norm::rms_scale(sum[0], K, eps), c = along[0] / (float)K * r;
        for (int k = threadIdx.x; k < K; k += kWaves * 64) {
            const float t_r = E::load(t + k) * r, e = E::load(d + k);
            float v = r * __builtin_fmaf(-t_r, c, e * gain[k]);
            if (dtotal.p) v += E::load(dtotal.p + m * dtotal.ld + k);
            E::store(dx.p + m * dx.ld + k, v);
            to[k] = __builtin_fmaf(e, t_r, to[k]);
        }
    }
}

// The sum of the work-groups' rows, 64 columns a work-group: sixteen waves take every sixteenth row each.
static __global__ __launch_bounds__(1024) void norm_gain_kernel(const float *__restrict__ partial, float *__restrict__ dgain,
                                                                int64_t rows, int K) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int64_t p = wave; p < rows; p += 16) s += partial[p * K + k];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || k >= K) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    dgain[k] = s;
}

}  // namespace jscan

// causal_conv_kernels.h - the short causal convolution in front of a scan: every channel over its own last W
// tokens (W = 2, 3, 4), its backward pass and its decode step.
//
//     v_t[d] = bias[d] + sum_{k < W} w[d][k] e_{t+k}[d],   y_t = act(v_t)
//     e = the W - 1 tokens of the starting state, then x_0, x_1, ...;  the state that goes out is e_n .. e_{n+W-2}
//     backward, with z_t = dy_t act'(v_t):
//     de_i = sum_k w[k] z_{i-k}  (+ the outgoing state's gradient at i >= n),   dw[k] = sum_t z_t e_{t+k},   db = sum_t z_t
//
// Memory bounds it: 4 bytes an element of bf16 (backward 6) for about 20 (30) instructions.  A thread keeps N
// channels' window of W - 1 tokens in registers and walks a run of tokens, so x is read once but for the
// W - 1 tokens before each run (backward: and the W - 1 behind it).
// Measured (bf16, four taps, SiLU; us, bytes that cross HBM over time): forward 16 x 4096 x 8192 359, 6.0 TB/s; 8 x
// 4096 x 8192 forward 193, 5.6, backward 288 + 5 for the sums, 5.7; step 256 x 8192 6.3 from the
// last-level cache.
#pragma once

#include <type_traits>

#include "activation.h"
#include "token_rows.h"

namespace jscan {

namespace conv {

constexpr int kThreads = 256;

// N channels of one token in memory: aligned to their element alone, so that any row stride takes the same
// loads (the hardware takes any address).
template <typename E, int N> struct Word;
template <> struct Word<BF16, 4> {
    typedef uint32_t raw __attribute__((ext_vector_type(2), aligned(2)));
    static __device__ __forceinline__ void unpack(raw w, float (&f)[4]) {
        f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[4]) {
        return raw{pack2(f[0], f[1]), pack2(f[2], f[3])};
    }
};
template <> struct Word<BF16, 2> {
    typedef uint32_t raw __attribute__((aligned(2)));
    static __device__ __forceinline__ void unpack(raw w, float (&f)[2]) { f[0] = bf16_lo(w), f[1] = bf16_hi(w); }
    static __device__ __forceinline__ raw pack(const float (&f)[2]) { return pack2(f[0], f[1]); }
};
template <> struct Word<BF16, 1> {
    using raw = uint16_t;
    static __device__ __forceinline__ void unpack(raw w, float (&f)[1]) { f[0] = bf16_bits_to_f32(w); }
    static __device__ __forceinline__ raw pack(const float (&f)[1]) { return f32_to_bf16_bits(f[0]); }
};
template <> struct Word<F32, 4> {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    static __device__ __forceinline__ void unpack(raw w, float (&f)[4]) {
        f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
    }
    static __device__ __forceinline__ raw pack(const float (&f)[4]) { return raw{f[0], f[1], f[2], f[3]}; }
};
template <> struct Word<F32, 2> {
    typedef float raw __attribute__((ext_vector_type(2), aligned(4)));
    static __device__ __forceinline__ void unpack(raw w, float (&f)[2]) { f[0] = w.x, f[1] = w.y; }
    static __device__ __forceinline__ raw pack(const float (&f)[2]) { return raw{f[0], f[1]}; }
};
template <> struct Word<F32, 1> {
    using raw = float;
    static __device__ __forceinline__ void unpack(raw w, float (&f)[1]) { f[0] = w; }
    static __device__ __forceinline__ raw pack(const float (&f)[1]) { return f[0]; }
};

// kNt: with the non-temporal hint, for tensors that go by.
template <typename E, int N, bool kNt = false>
__device__ __forceinline__ typename Word<E, N>::raw load(const typename E::store_t *p) {
    if constexpr (kNt) return __builtin_nontemporal_load(reinterpret_cast<const typename Word<E, N>::raw *>(p));
    return *reinterpret_cast<const typename Word<E, N>::raw *>(p);
}
template <typename E, int N, bool kNt = false>
__device__ __forceinline__ void store(typename E::store_t *p, typename Word<E, N>::raw v) {
    if constexpr (kNt) __builtin_nontemporal_store(v, reinterpret_cast<typename Word<E, N>::raw *>(p));
    else *reinterpret_cast<typename Word<E, N>::raw *>(p) = v;
}

// How a call is dealt out: `lanes` (a power of two) lanes side by side take N channels each, the work-group's
// kThreads / lanes rows of lanes take runs of `run` tokens one after the other, `segs` work-groups a sequence.
struct Split {
    int lanes_log, strips, segs;
    int64_t run;
};

// A thread's channels and tokens.  The last word of a row reaches back over the one before it where N does not
// divide D: both compute the same values.
template <int N> struct Place {
    int64_t b, t0;
    int strip, seg, row, col, c0;   // strip, work-group of the sequence, row of lanes, lane, first channel
    bool active;
    // near: consecutive work-groups to one XCD (ids 8 apart), so that the tokens around a run are in its L2.
    __device__ __forceinline__ Place(const Split &sp, int D, bool near) {
        const uint32_t per = gridDim.x / 8, id = blockIdx.x;
        const uint32_t v = near && id < per * 8 ? (id % 8) * per + id / 8 : id;
        const uint32_t rest = v / sp.strips;
        strip = v % sp.strips;
        seg = rest % sp.segs;
        b = rest / sp.segs;
        col = threadIdx.x & ((1 << sp.lanes_log) - 1);
        row = threadIdx.x >> sp.lanes_log;
        const int word = (strip << sp.lanes_log) + col;
        active = word * N < D;
        c0 = min(word * N, D - N);
        t0 = ((int64_t)seg * (kThreads >> sp.lanes_log) + row) * sp.run;
    }
};

template <int W, int N> struct Taps {
    float w[W][N], bias[N];
    __device__ __forceinline__ Taps(const float *wp, const float *bp, int c0) {
#pragma unroll
        for (int v = 0; v < N; ++v) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][v] = wp[(int64_t)(c0 + v) * W + k];
            bias[v] = bp ? bp[c0 + v] : 0.0f;
        }
    }
};

// The window of the W - 1 tokens before token t0: the starting state's (zeros without one) or x's.
template <typename E, int N, int W>
__device__ __forceinline__ void load_window(typename Word<E, N>::raw (&win)[W - 1], TokenRows<const typename E::store_t> x,
                                            const typename E::store_t *state, int64_t b, int64_t L, int D, int64_t t0,
                                            int c0) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (t0 == 0) {
            win[j] = state ? load<E, N>(state + (b * (W - 1) + j) * D + c0) : typename Word<E, N>::raw{};
        } else {
            win[j] = load<E, N>(x.p + (b * L + t0 - (W - 1) + j) * x.ld + c0);
        }
    }
}

}  // namespace conv

// Tokens that are on their way while as many are computed.
constexpr int kForwardStage = 8, kBackwardStage = 4;

template <typename E, int N, int W, Act A, bool kNt>
__global__ __launch_bounds__(conv::kThreads) void causal_conv_kernel(
    TokenRows<const typename E::store_t> x, const typename E::store_t *state, const float *__restrict__ w,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, TokenRows<typename E::store_t> y,
    typename E::store_t *state_out, int64_t L, int D, conv::Split sp) {
    using raw = typename conv::Word<E, N>::raw;
    constexpr int U = kForwardStage;
    const conv::Place<N> at(sp, D, true);
    if (!at.active || (at.t0 >= L && at.t0 > 0)) return;   // an empty sequence still hands its state on
    const int64_t n = tokens_of(lengths, at.b, L), t0 = at.t0;
    raw win[W - 1];
    if (t0 < n || t0 == 0) conv::load_window<E, N, W>(win, x, state, at.b, L, D, t0, at.c0);
    if (t0 == 0 && state_out) {   // state may be state_out itself: only this thread reads and writes these channels
        raw tail[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t i = n + j;
            tail[j] = i < W - 1 ? win[0] : conv::load<E, N>(x.p + (at.b * L + i - (W - 1)) * x.ld + at.c0);
#pragma unroll
            for (int k = 1; k < W - 1; ++k)
                if (i == k) tail[j] = win[k];
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) conv::store<E, N>(state_out + (at.b * (W - 1) + j) * D + at.c0, tail[j]);
    }
    const int64_t end = min(t0 + sp.run, L), live = min(end, n);
    typename E::store_t *yp = y.p + (at.b * L + t0) * y.ld + at.c0;
    if (t0 < live) {
        const conv::Taps<W, N> taps(w, bias, at.c0);
        float e[W - 1][N];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) conv::Word<E, N>::unpack(win[j], e[j]);
        const typename E::store_t *xp = x.p + (at.b * L + t0) * x.ld + at.c0;
        const int64_t count = live - t0;
        raw next[U];
        auto fetch = [&](int64_t i0) {   // tokens behind the run's end read its last one
            if (i0 + U <= count) {
#pragma unroll
                for (int i = 0; i < U; ++i) next[i] = conv::load<E, N, kNt>(xp + i0 * x.ld + i * x.ld);
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i) next[i] = conv::load<E, N, kNt>(xp + min(i0 + i, count - 1) * x.ld);
            }
        };
        auto block = [&](auto ends_c, int64_t i0) {   // U tokens; fewer at the run's end
            constexpr bool ends = decltype(ends_c)::value;
            raw cur[U];
#pragma unroll
            for (int i = 0; i < U; ++i) cur[i] = next[i];
            if (!ends && i0 + U < count) fetch(i0 + U);
            float ew[W - 1 + U][N];
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < N; ++v) ew[j][v] = e[j][v];
            typename E::store_t *dst = yp + i0 * y.ld;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float o[N];
                conv::Word<E, N>::unpack(cur[i], ew[W - 1 + i]);
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    float s = taps.bias[v];
#pragma unroll
                    for (int k = 0; k < W; ++k) s = __builtin_fmaf(taps.w[k][v], ew[i + k][v], s);
                    o[v] = activate<A>(s);
                }
                if (!ends || i0 + i < count) conv::store<E, N, kNt>(dst + i * y.ld, conv::Word<E, N>::pack(o));
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < N; ++v) e[j][v] = ew[U + j][v];
        };
        fetch(0);
        int64_t i0 = 0;
        for (; i0 + U <= count; i0 += U) block(std::false_type{}, i0);
        if (i0 < count) block(std::true_type{}, i0);
    }
    for (int64_t t = max(t0, n); t < end; ++t) conv::store<E, N>(yp + (t - t0) * y.ld, raw{});
}

// The backward pass.  At token t a thread has z_t and the W - 1 before it, which give the gradient of token
// t - (W - 1); W - 1 tokens behind the run complete its own.  Gradients of taps and bias are summed over the
// run in registers, over the work-group's runs in LDS and over work-groups by conv_sum_kernel: fixed
// orders, so results repeat bit for bit.  partial[sequence and work-group][W + 1][D].
template <typename E, int N, int W, Act A, bool kNt>
__global__ __launch_bounds__(conv::kThreads) void causal_conv_backward_kernel(
    TokenRows<const typename E::store_t> x, const typename E::store_t *__restrict__ state, const float *__restrict__ w,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, TokenRows<const typename E::store_t> dy,
    const typename E::store_t *__restrict__ dstate_out, TokenRows<typename E::store_t> dx,
    typename E::store_t *__restrict__ dstate, float *__restrict__ partial, int64_t L, int D, conv::Split sp) {
    using raw = typename conv::Word<E, N>::raw;
    constexpr int U = kBackwardStage;
    __shared__ float sums[(W + 1) * N * conv::kThreads];
    const conv::Place<N> at(sp, D, !kNt);
    float dw[W + 1][N];   // taps, then bias
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int v = 0; v < N; ++v) dw[k][v] = 0.0f;

    const int64_t t0 = at.t0;
    if (at.active && (t0 < L || t0 == 0)) {
        const int64_t n = tokens_of(lengths, at.b, L), end = min(t0 + sp.run, L), live = min(end, n);
        typename E::store_t *dxp = dx.p + at.b * L * dx.ld + at.c0;
        if (t0 < live || t0 == 0) {
            const conv::Taps<W, N> taps(w, bias, at.c0);
            raw win[W - 1];
            conv::load_window<E, N, W>(win, x, state, at.b, L, D, t0, at.c0);
            float e[W - 1][N], z[W - 1][N];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                conv::Word<E, N>::unpack(win[j], e[j]);
#pragma unroll
                for (int v = 0; v < N; ++v) z[j][v] = 0.0f;
            }
            const typename E::store_t *xp = x.p + at.b * L * x.ld + at.c0, *dyp = dy.p + at.b * L * dy.ld + at.c0;
            const int64_t first = t0 == 0 ? -(W - 1) : t0;   // the first gradient that this run writes
            const int64_t stop = live + W - 1;               // tokens from which its gradients come
            raw nx[U], ny[U];
            auto fetch = [&](int64_t t) {   // tokens behind the sequence read its last one
                if (t + U <= n) {
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        nx[i] = conv::load<E, N, kNt>(xp + t * x.ld + i * x.ld);
                        ny[i] = conv::load<E, N, kNt>(dyp + t * dy.ld + i * dy.ld);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int64_t c = min(t + i, n - 1);
                        nx[i] = conv::load<E, N, kNt>(xp + c * x.ld);
                        ny[i] = conv::load<E, N, kNt>(dyp + c * dy.ld);
                    }
                }
            };
            // U tokens from t.  Whole blocks are the run's own; what is left of it, and the tokens behind it, go
            // token by token (`ends`), z zero behind the sequence.
            auto block = [&](auto ends_c, int64_t t) {
                constexpr bool ends = decltype(ends_c)::value;
                raw cx[U], cy[U];
#pragma unroll
                for (int i = 0; i < U; ++i) cx[i] = nx[i], cy[i] = ny[i];
                if (t + U < (ends ? min(stop, n) : stop)) fetch(t + U);
                float ew[W - 1 + U][N], zw[W - 1 + U][N];   // windows over the block
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int v = 0; v < N; ++v) ew[j][v] = e[j][v], zw[j][v] = z[j][v];
                typename E::store_t *dst = dxp + t * dx.ld;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (ends && t + i >= stop) return;
                    float g[N];
                    conv::Word<E, N>::unpack(cx[i], ew[W - 1 + i]);
                    conv::Word<E, N>::unpack(cy[i], zw[W - 1 + i]);
#pragma unroll
                    for (int v = 0; v < N; ++v) {
                        float zt = zw[W - 1 + i][v];
                        if constexpr (A == Act::Silu) {
                            float s = taps.bias[v];
#pragma unroll
                            for (int k = 0; k < W; ++k) s = __builtin_fmaf(taps.w[k][v], ew[i + k][v], s);
                            zt *= silu_slope(s);
                        }
                        if (ends) zt = t + i < n ? zt : 0.0f;
                        zw[W - 1 + i][v] = zt;
                        if (!ends || t + i < live) {
#pragma unroll
                            for (int k = 0; k < W; ++k) dw[k][v] = __builtin_fmaf(zt, ew[i + k][v], dw[k][v]);
                            dw[W][v] += zt;
                        }
                        g[v] = taps.w[0][v] * zt;   // of token t + i - (W - 1), of whose z this is the last
#pragma unroll
                        for (int k = 1; k < W; ++k) g[v] = __builtin_fmaf(taps.w[k][v], zw[W - 1 + i - k][v], g[v]);
                    }
                    const int64_t s = t + i - (W - 1);
                    if ((ends || i < W - 1) && s < first) continue;
                    if (ends && t + i >= n && dstate_out) {   // a token of the outgoing state
                        float f[N];
                        conv::Word<E, N>::unpack(conv::load<E, N>(dstate_out + (at.b * (W - 1) + t + i - n) * D + at.c0), f);
#pragma unroll
                        for (int v = 0; v < N; ++v) g[v] += f[v];
                    }
                    if (!(ends || i < W - 1) || s >= 0)
                        conv::store<E, N, kNt>(dst + (i - (W - 1)) * dx.ld, conv::Word<E, N>::pack(g));
                    else if (dstate)
                        conv::store<E, N>(dstate + (at.b * (W - 1) + t + i) * D + at.c0, conv::Word<E, N>::pack(g));
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int v = 0; v < N; ++v) e[j][v] = ew[U + j][v], z[j][v] = zw[U + j][v];
            };
            if (t0 < n) fetch(t0);
            int64_t t = t0;
            for (; t + U <= live; t += U) block(std::false_type{}, t);
            for (; t < stop; t += U) block(std::true_type{}, t);
        }
        for (int64_t t = max(t0, n); t < end; ++t) conv::store<E, N>(dxp + t * dx.ld, raw{});
    }

    const int lanes = 1 << sp.lanes_log, rows = conv::kThreads >> sp.lanes_log, across = lanes * N;
    // sums[k][row][channel of the strip]
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int v = 0; v < N; ++v) sums[(k * rows + at.row) * across + at.col * N + v] = dw[k][v];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * across; i += conv::kThreads) {
        const int k = i / across, c = i % across, word = (at.strip << sp.lanes_log) + c / N;
        if (word * N >= D) continue;
        float s = 0.0f;
        for (int r = 0; r < rows; ++r) s += sums[(k * rows + r) * across + c];
        partial[((at.b * sp.segs + at.seg) * (W + 1) + k) * D + min(word * N, D - N) + c % N] = s;
    }
}

// The sums of the work-groups' shares, 64 channels of one tap (or of the bias) a work-group: sixteen waves take every
// sixteenth share each.
template <int W>
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float *__restrict__ partial, float *__restrict__ dw,
                                                        float *__restrict__ dbias, int64_t shares, int D) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.y;
    const int d = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (d < D) {
#pragma unroll 8
        for (int64_t p = wave; p < shares; p += 16) s += partial[(p * (W + 1) + k) * D + d];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || d >= D) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    if (k < W) dw[(int64_t)d * W + k] = s;
    else if (dbias) dbias[d] = s;
}

// One decode token: a thread has N channels of kRows sequences, one set of taps for them all.  A missing last
// sequence reads the one before it and stores nothing.
template <typename E, int N, int W, Act A, int kRows>
__global__ __launch_bounds__(conv::kThreads) void causal_conv_step_kernel(
    typename E::store_t *__restrict__ state, const typename E::store_t *__restrict__ x, const float *__restrict__ w,
    const float *__restrict__ bias, typename E::store_t *__restrict__ y, int64_t batch, int D, int words, int64_t ld_x,
    int64_t ld_y) {
    using raw = typename conv::Word<E, N>::raw;
    const int64_t id = (int64_t)blockIdx.x * conv::kThreads + threadIdx.x, b0 = id / words * kRows;
    if (b0 >= batch) return;
    const int c0 = (int)(id % words) * N;
    raw win[kRows][W];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t b = min(b0 + r, batch - 1);
        const typename E::store_t *st = state + b * (W - 1) * D + c0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[r][j] = conv::load<E, N>(st + (int64_t)j * D);
        win[r][W - 1] = conv::load<E, N>(x + b * ld_x + c0);
    }
    const conv::Taps<W, N> taps(w, bias, c0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t b = b0 + r;
        if (b >= batch) break;
        float o[N];
#pragma unroll
        for (int v = 0; v < N; ++v) o[v] = taps.bias[v];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            float f[N];
            conv::Word<E, N>::unpack(win[r][k], f);
#pragma unroll
            for (int v = 0; v < N; ++v) o[v] = __builtin_fmaf(taps.w[k][v], f[v], o[v]);
        }
#pragma unroll
        for (int v = 0; v < N; ++v) o[v] = activate<A>(o[v]);
        typename E::store_t *st = state + b * (W - 1) * D + c0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) conv::store<E, N>(st + (int64_t)j * D, win[r][j + 1]);
        conv::store<E, N>(y + b * ld_y + c0, conv::Word<E, N>::pack(o));
    }
}

}  // namespace jscan

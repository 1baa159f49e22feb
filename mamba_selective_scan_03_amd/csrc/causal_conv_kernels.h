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
        return raw{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
    }
};
template <> struct Word<BF16, 8> {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    static __device__ __forceinline__ void unpack(raw w, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[8]) {
        return raw{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
    }
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
template <> struct Word<F32, 1> {
    using raw = float;
    static __device__ __forceinline__ void unpack(raw w, float (&f)[1]) { f[0] = w; }
    static __device__ __forceinline__ raw pack(const float (&f)[1]) { return f[0]; }
};

template <typename E, int N> __device__ __forceinline__ typename Word<E, N>::raw load(const typename E::store_t *p) {
    return *reinterpret_cast<const typename Word<E, N>::raw *>(p);
}
template <typename E, int N>
__device__ __forceinline__ void store(typename E::store_t *p, typename Word<E, N>::raw v) {
    *reinterpret_cast<typename Word<E, N>::raw *>(p) = v;
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
    __device__ __forceinline__ Place(const Split &sp, int D) {
        // consecutive work-groups to one XCD (ids 8 apart): the tokens before a run are in its L2
        const uint32_t per = gridDim.x / 8, id = blockIdx.x;
        const uint32_t v = id < per * 8 ? (id % 8) * per + id / 8 : id;
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

constexpr int kConvStage = 8;   // tokens that are on their way while as many are computed

template <typename E, int N, int W, Act A>
__global__ __launch_bounds__(conv::kThreads) void causal_conv_kernel(
    TokenRows<const typename E::store_t> x, const typename E::store_t *state, const float *__restrict__ w,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, TokenRows<typename E::store_t> y,
    typename E::store_t *state_out, int64_t L, int D, conv::Split sp) {
    using raw = typename conv::Word<E, N>::raw;
    constexpr int U = kConvStage;
    const conv::Place<N> at(sp, D);
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
                for (int i = 0; i < U; ++i) next[i] = conv::load<E, N>(xp + (i0 + i) * x.ld);
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i) next[i] = conv::load<E, N>(xp + min(i0 + i, count - 1) * x.ld);
            }
        };
        fetch(0);
        for (int64_t i0 = 0; i0 < count; i0 += U) {
            raw cur[U];
#pragma unroll
            for (int i = 0; i < U; ++i) cur[i] = next[i];
            if (i0 + U < count) fetch(i0 + U);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float f[N], o[N];
                conv::Word<E, N>::unpack(cur[i], f);
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    float s = taps.bias[v];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) s = __builtin_fmaf(taps.w[k][v], e[k][v], s);
                    o[v] = activate<A>(__builtin_fmaf(taps.w[W - 1][v], f[v], s));
#pragma unroll
                    for (int k = 0; k < W - 2; ++k) e[k][v] = e[k + 1][v];
                    e[W - 2][v] = f[v];
                }
                if (i0 + i < count) conv::store<E, N>(yp + (i0 + i) * y.ld, conv::Word<E, N>::pack(o));
            }
        }
    }
    for (int64_t t = max(t0, n); t < end; ++t) conv::store<E, N>(yp + (t - t0) * y.ld, raw{});
}

// The backward pass.  At token t a thread has z_t and the W - 1 before it, which give the gradient of token
// t - (W - 1); W - 1 tokens behind the run complete its own.  Gradients of taps and bias are summed over the
// run in registers, over the work-group's runs in LDS and over work-groups by conv_sum_kernel: fixed
// orders, so results repeat bit for bit.  partial[sequence and work-group][W + 1][D].
template <typename E, int N, int W, Act A>
__global__ __launch_bounds__(conv::kThreads) void causal_conv_backward_kernel(
    TokenRows<const typename E::store_t> x, const typename E::store_t *__restrict__ state, const float *__restrict__ w,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, TokenRows<const typename E::store_t> dy,
    const typename E::store_t *__restrict__ dstate_out, TokenRows<typename E::store_t> dx,
    typename E::store_t *__restrict__ dstate, float *__restrict__ partial, int64_t L, int D, conv::Split sp) {
    using raw = typename conv::Word<E, N>::raw;
    constexpr int U = kConvStage;
    __shared__ float sums[(W + 1) * N * conv::kThreads];
    const conv::Place<N> at(sp, D);
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
            // the gradient of token s from z_s .. z_{s+W-1}, of which zt is the last
            auto out = [&](int64_t s, const float (&zt)[N]) {
                float g[N];
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    g[v] = taps.w[0][v] * zt[v];
#pragma unroll
                    for (int k = 1; k < W; ++k) g[v] = __builtin_fmaf(taps.w[k][v], z[W - 1 - k][v], g[v]);
                }
                if (s < first) return;
                if (s + (W - 1) >= n && dstate_out) {
                    float f[N];
                    conv::Word<E, N>::unpack(
                        conv::load<E, N>(dstate_out + (at.b * (W - 1) + s + (W - 1) - n) * D + at.c0), f);
#pragma unroll
                    for (int v = 0; v < N; ++v) g[v] += f[v];
                }
                if (s >= 0) conv::store<E, N>(dxp + s * dx.ld, conv::Word<E, N>::pack(g));
                else if (dstate) conv::store<E, N>(dstate + (at.b * (W - 1) + s + (W - 1)) * D + at.c0, conv::Word<E, N>::pack(g));
            };
            auto shift = [&](const float (&zt)[N]) {
#pragma unroll
                for (int v = 0; v < N; ++v) {
#pragma unroll
                    for (int k = 0; k < W - 2; ++k) z[k][v] = z[k + 1][v];
                    z[W - 2][v] = zt[v];
                }
            };
            // one token: z_t, its share of the taps' gradients where it is the run's own
            auto token = [&](int64_t t, raw xw, raw dyw, bool mine) {
                float f[N], zt[N];
                conv::Word<E, N>::unpack(xw, f);
                conv::Word<E, N>::unpack(dyw, zt);
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    if constexpr (A == Act::Silu) {
                        float s = taps.bias[v];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) s = __builtin_fmaf(taps.w[k][v], e[k][v], s);
                        zt[v] *= silu_slope(__builtin_fmaf(taps.w[W - 1][v], f[v], s));
                    }
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][v] = __builtin_fmaf(zt[v], e[k][v], dw[k][v]);
                        dw[W - 1][v] = __builtin_fmaf(zt[v], f[v], dw[W - 1][v]);
                        dw[W][v] += zt[v];
                    }
#pragma unroll
                    for (int k = 0; k < W - 2; ++k) e[k][v] = e[k + 1][v];
                    e[W - 2][v] = f[v];
                }
                out(t - (W - 1), zt);
                shift(zt);
            };
            raw nx[U], ny[U];
            auto fetch = [&](int64_t t) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int64_t c = min(t + i, live - 1);
                    nx[i] = conv::load<E, N>(xp + c * x.ld);
                    ny[i] = conv::load<E, N>(dyp + c * dy.ld);
                }
            };
            if (t0 < live) fetch(t0);
            for (int64_t t = t0; t < live; t += U) {
                raw cx[U], cy[U];
#pragma unroll
                for (int i = 0; i < U; ++i) cx[i] = nx[i], cy[i] = ny[i];
                if (t + U < live) fetch(t + U);
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (t + i < live) token(t + i, cx[i], cy[i], true);
            }
            for (int64_t t = live; t < live + W - 1; ++t) {   // behind the run: zero behind the sequence's end
                if (t < n) {
                    token(t, conv::load<E, N>(xp + t * x.ld), conv::load<E, N>(dyp + t * dy.ld), false);
                } else {
                    const float zero[N] = {};
                    out(t - (W - 1), zero);
                    shift(zero);
                }
            }
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

// The sums of the work-groups' shares, 64 channels of one tap (or of the bias) a work-group: four waves take
// every fourth share each.
template <int W>
__global__ __launch_bounds__(256) void conv_sum_kernel(const float *__restrict__ partial, float *__restrict__ dw,
                                                       float *__restrict__ dbias, int64_t shares, int D) {
    __shared__ float part[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.y;
    const int d = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (d < D) {
#pragma unroll 8
        for (int64_t p = wave; p < shares; p += 4) s += partial[(p * (W + 1) + k) * D + d];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || d >= D) return;
    s = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    if (k < W) dw[(int64_t)d * W + k] = s;
    else if (dbias) dbias[d] = s;
}

// One decode token: a thread has N channels of one sequence.
template <typename E, int N, int W, Act A>
__global__ __launch_bounds__(conv::kThreads) void causal_conv_step_kernel(
    typename E::store_t *__restrict__ state, const typename E::store_t *__restrict__ x, const float *__restrict__ w,
    const float *__restrict__ bias, typename E::store_t *__restrict__ y, int64_t batch, int D, int words, int64_t ld_x,
    int64_t ld_y) {
    using raw = typename conv::Word<E, N>::raw;
    const int64_t id = (int64_t)blockIdx.x * conv::kThreads + threadIdx.x, b = id / words;
    if (b >= batch) return;
    const int c0 = (int)(id - b * words) * N;
    typename E::store_t *st = state + b * (W - 1) * D + c0;
    raw win[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = conv::load<E, N>(st + (int64_t)j * D);
    win[W - 1] = conv::load<E, N>(x + b * ld_x + c0);
    const conv::Taps<W, N> taps(w, bias, c0);
    float o[N];
#pragma unroll
    for (int v = 0; v < N; ++v) o[v] = taps.bias[v];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float f[N];
        conv::Word<E, N>::unpack(win[k], f);
#pragma unroll
        for (int v = 0; v < N; ++v) o[v] = __builtin_fmaf(taps.w[k][v], f[v], o[v]);
    }
#pragma unroll
    for (int v = 0; v < N; ++v) o[v] = activate<A>(o[v]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) conv::store<E, N>(st + (int64_t)j * D, win[j + 1]);
    conv::store<E, N>(y + b * ld_y + c0, conv::Word<E, N>::pack(o));
}

}  // namespace jscan

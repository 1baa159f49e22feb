// gated_scan_kernels.h - the gated recurrence over whole sequences, its backward pass and its
// decode step (gated_update.h has the mathematics).
#pragma once

#include "gated_update.h"

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

// One lane per (sequence, channel), tokens in order.
template <typename E, GateForm F>
__global__ __launch_bounds__(64) void gated_lane_kernel(TokenRows<const typename E::store_t> g,
                                                        TokenRows<const typename E::store_t> u,
                                                        const float *__restrict__ h0,
                                                        const int32_t *__restrict__ lengths,
                                                        TokenRows<typename E::store_t> y, float *h_final, int64_t L,
                                                        int D, int strips) {
    const int64_t b = blockIdx.x / strips;
    const int d = (int)(blockIdx.x % strips) * 64 + threadIdx.x;
    if (d >= D) return;
    const int64_t n = tokens_of(lengths, b, L);
    float h = h0 ? h0[b * D + d] : 0.0f;
    for (int64_t t = 0; t < n; ++t) {
        const int64_t row = b * L + t;
        const Gate k = gate<F>(E::load(g.p + row * g.ld + d));
        h = gated_advance(h, k.a, gated_input<F>(k, E::load(u.p + row * u.ld + d)));
        E::store(y.p + row * y.ld + d, h);
    }
    for (int64_t t = n; t < L; ++t) E::store(y.p + (b * L + t) * y.ld + d, 0.0f);
    h_final[b * D + d] = h;
}

template <typename E, GateForm F>
__global__ __launch_bounds__(64) void gated_lane_backward_kernel(
    TokenRows<const typename E::store_t> g, TokenRows<const typename E::store_t> u,
    TokenRows<const typename E::store_t> y, TokenRows<const typename E::store_t> dy, const float *__restrict__ h0,
    const float *dh_final, const int32_t *__restrict__ lengths, TokenRows<typename E::store_t> dg,
    TokenRows<typename E::store_t> du, float *dh0, int64_t L, int D, int strips) {
    const int64_t b = blockIdx.x / strips;
    const int d = (int)(blockIdx.x % strips) * 64 + threadIdx.x;
    if (d >= D) return;
    const int64_t n = tokens_of(lengths, b, L);
    float c = dh_final ? dh_final[b * D + d] : 0.0f;
    for (int64_t t = L - 1; t >= n; --t) {
        E::store(dg.p + (b * L + t) * dg.ld + d, 0.0f);
        E::store(du.p + (b * L + t) * du.ld + d, 0.0f);
    }
    for (int64_t t = n - 1; t >= 0; --t) {
        const int64_t row = b * L + t;
        const Gate k = gate<F>(E::load(g.p + row * g.ld + d));
        const float h = t > 0 ? E::load(y.p + (row - 1) * y.ld + d) : (h0 ? h0[b * D + d] : 0.0f);
        const float G = E::load(dy.p + row * dy.ld + d) + c;
        c = k.a * G;
        if constexpr (F == GateForm::Decay) {
            E::store(dg.p + row * dg.ld + d, c * h);
            E::store(du.p + row * du.ld + d, G);
        } else {
            E::store(dg.p + row * dg.ld + d, c * k.b * (h - E::load(u.p + row * u.ld + d)));
            E::store(du.p + row * du.ld + d, k.b * G);
        }
    }
    if (dh0) dh0[b * D + d] = c;
}

// One decode token: one thread per (sequence, channel), the state in place.
template <typename E, GateForm F>
__global__ __launch_bounds__(256) void gated_step_kernel(float *__restrict__ h, const typename E::store_t *g,
                                                         const typename E::store_t *u, typename E::store_t *y, int D,
                                                         int blocks_per_row, int64_t ld_g, int64_t ld_u,
                                                         int64_t ld_y) {
    const int64_t b = blockIdx.x / blocks_per_row;
    const int d = (int)(blockIdx.x % blocks_per_row) * 256 + threadIdx.x;
    if (d >= D) return;
    const Gate k = gate<F>(E::load(g + b * ld_g + d));
    const float v = gated_advance(h[b * D + d], k.a, gated_input<F>(k, E::load(u + b * ld_u + d)));
    h[b * D + d] = v;
    E::store(y + b * ld_y + d, v);
}

}  // namespace jscan

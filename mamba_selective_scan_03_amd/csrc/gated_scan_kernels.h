// gated_scan_kernels.h - the gated recurrence over whole sequences, its backward pass and its
// decode step (gated_update.h has the mathematics).
//
// Both directions are the affine scan s <- a s + x of one fp32 state per channel:
//     forward    s = h,  x = b u,     tokens in order
//     backward   s = c,  x = a dy,    tokens from the last to the first (c_t = a_t (dy_t + c_{t+1}))
// They move 6 (fp32: 12) and 10 to 12 (20 to 24) bytes per element for a dozen instructions, so memory bounds
// them: every byte should move once, and enough of them at a time, although one channel's tokens
// depend on each other.
//
// Work-group: a strip of LC lanes x V::n channels over all tokens of one sequence (or of one segment of it, see
// below).  Its S = 64 NW / LC thread rows take consecutive runs of TT tokens, a block of S TT tokens at a
// time, and the next block's words are on their way while one block is computed:
//   1. every thread composes its run's map s -> A s + H, keeping the maps (A_i, H_i) of its prefixes;
//   2. the runs' maps go through LDS; a thread carries the block's starting state through the maps
//      of the runs before its own (through lane shuffles first for the runs inside a wave);
//   3. the states are s_i = A_i s_in + H_i, independent of each other.
// Every order is fixed, so results repeat bit for bit.
//
// A run of eight tokens keeps two blocks of words and the maps of one in registers; sixteen tokens took the
// registers of the prefetch, four made twice the barriers.  Keeping (A_i, H_i) instead of walking the run a
// second time costs a multiply per element and makes the second pass independent.  Eight waves: sixteen ran
// the same where strips are many and lose registers to the backward pass (8 x 4096 x 8192 decay: scan 302
// us with sixteen, 307 us with eight; backward 515 and 513 us).  The gate is evaluated once; the maps are
// not rounded.
#pragma once

#include <type_traits>

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

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// What a lane loads and stores at a time: n channels in one word (their fp32 states in one state_word).  The
// two-channel bf16 word needs rows that start on 4 bytes and an even D; the one-channel word takes the rest.
struct Bf16x2 {
    using store_t = uint16_t;
    using word = uint32_t;
    using state_word = f32x2_t;
    static constexpr int n = 2;
    static __device__ __forceinline__ void unpack(word w, float (&f)[2]) {
        f[0] = bf16_lo(w);
        f[1] = bf16_hi(w);
    }
    static __device__ __forceinline__ word pack(const float (&f)[2]) { return pack_bf16x2(f[0], f[1]); }
};
struct Bf16x1 {
    using store_t = uint16_t;
    using word = uint16_t;
    using state_word = float;
    static constexpr int n = 1;
    static __device__ __forceinline__ void unpack(word w, float (&f)[1]) { f[0] = bf16_bits_to_f32(w); }
    static __device__ __forceinline__ word pack(const float (&f)[1]) { return f32_to_bf16_bits(f[0]); }
};
struct F32x1 {
    using store_t = float;
    using word = float;
    using state_word = float;
    static constexpr int n = 1;
    static __device__ __forceinline__ void unpack(word w, float (&f)[1]) { f[0] = w; }
    static __device__ __forceinline__ word pack(const float (&f)[1]) { return f[0]; }
};

// A sequence's tokens cut into n_seg segments of seg_len tokens of scan order (n_seg = 1: not cut).
// sums[b][seg][D] holds the segments' maps (A, H), start[b][D] a copy of the scan's starting state (the caller's
// own array may be overwritten by the final one while late segments still need it).
struct SegSplit {
    int n_seg;
    int64_t seg_len;
    float2 *sums;
    float *start;
};

namespace strip {

// A wave's place in its work-group and a lane's in its strip.
template <typename V, int LC, int NW, int TT> struct Place {
    static constexpr int kSub = 64 / LC;         // runs per wave
    static constexpr int kRuns = kSub * NW;      // runs per work-group
    static constexpr int kBlock = kRuns * TT;    // tokens per block
};

// One tensor's rows as a strip walks them in scan order (kRev: from the last token down).  A row's address
// is a wave-uniform part and a 32-bit lane part (channel, and the lane's run inside the wave).  kNt: whole
// blocks go by with the non-temporal hint.
template <typename V, int LC, int TT, bool kRev, bool kNt> struct Stream {
    using word = typename V::word;
    char *base;          // row of token 0 of the sequence, channel 0
    int64_t ld;          // bytes between rows
    uint32_t lane_off;   // channel and run part of the address
    uint32_t chan_off;   // channel part alone

    template <typename T>
    __device__ __forceinline__ Stream(TokenRows<T> r, int64_t b, int64_t L, int sub, uint32_t channel_word) {
        ld = r.ld * (int64_t)sizeof(typename V::store_t);
        base = reinterpret_cast<char *>(const_cast<typename V::store_t *>(r.p)) + b * L * ld;
        chan_off = channel_word * (uint32_t)sizeof(word);
        const int runs_down = kRev ? 64 / LC - 1 - sub : sub;
        lane_off = chan_off + (uint32_t)(runs_down * TT) * (uint32_t)ld;
    }
    // Row address of step i of the wave's runs, which start at scan position tau (of n): the lowest
    // token among the wave's lanes.
    __device__ __forceinline__ char *row(int64_t tau, int64_t n, int i) const {
        const int64_t t = kRev ? n - 1 - tau - i - (64 / LC - 1) * TT : tau + i;
        return base + t * ld;
    }
    __device__ __forceinline__ void load(word (&w)[TT], int64_t tau, int64_t n, int shift) const {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const word *p = reinterpret_cast<const word *>(row(tau, n, i) + shift * ld + lane_off);
            if constexpr (kNt) w[i] = __builtin_nontemporal_load(p);
            else w[i] = *p;
        }
    }
    // The same near the ends: token by token, tokens outside [lo, hi] taken at the nearer end.
    __device__ __forceinline__ void load_clamped(word (&w)[TT], int64_t lane_tau, int64_t n, int shift, int64_t lo,
                                                 int64_t hi) const {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            int64_t t = (kRev ? n - 1 - lane_tau - i : lane_tau + i) + shift;
            t = t < lo ? lo : (t > hi ? hi : t);
            w[i] = *reinterpret_cast<const word *>(base + t * ld + chan_off);
        }
    }
    __device__ __forceinline__ void store(word v, int64_t tau, int64_t n, int i) const {
        word *p = reinterpret_cast<word *>(row(tau, n, i) + lane_off);
        if constexpr (kNt) __builtin_nontemporal_store(v, p);
        else *p = v;
    }
    __device__ __forceinline__ void store_at(word v, int64_t t) const {
        *reinterpret_cast<word *>(base + t * ld + chan_off) = v;
    }
};

// The saved fp32 states [batch][rows][D]: row r of a sequence is the state before its token r TT, where one thread's
// run starts in the forward scan.  A row's address is a wave-uniform part and a 32-bit lane part, as in Stream.
template <typename V, int LC, int TT, bool kRev, bool kNt> struct Starts {
    using word = typename V::state_word;
    char *base;          // row 0 of the sequence, channel 0
    int64_t ld;          // bytes between rows
    uint32_t lane_off, chan_off;

    __device__ __forceinline__ Starts(float *p, int64_t b, int64_t L, int D, int sub, uint32_t channel_word) {
        ld = (int64_t)D * 4;
        base = reinterpret_cast<char *>(p) + b * ((L + TT - 1) / TT) * ld;
        chan_off = channel_word * (uint32_t)sizeof(word);
        lane_off = chan_off + (uint32_t)(kRev ? 64 / LC - 1 - sub : sub) * (uint32_t)ld;
    }
    // Row of the wave's run with the lowest token (the wave's runs start at scan position tau, whose last token,
    // of `top`, is a run's end where kRev).
    __device__ __forceinline__ word *row(int64_t tau, int64_t top) const {
        const int64_t r = kRev ? (top - tau) / TT - 64 / LC : tau / TT;
        return reinterpret_cast<word *>(base + r * ld + lane_off);
    }
    __device__ __forceinline__ void load(float (&s)[V::n], int64_t tau, int64_t top) const {
        const word *p = row(tau, top);
        unpack(kNt ? __builtin_nontemporal_load(p) : *p, s);
    }
    // The state before the run that holds scan position lane_tau first; runs behind the scan's end take row 0.
    __device__ __forceinline__ void load_clamped(float (&s)[V::n], int64_t lane_tau, int64_t top) const {
        const int64_t r = (top - lane_tau) / TT - 1;
        unpack(*reinterpret_cast<const word *>(base + (r < 0 ? 0 : r) * ld + chan_off), s);
    }
    __device__ __forceinline__ void store(const float (&s)[V::n], int64_t tau) const {
        word w;
        if constexpr (V::n == 1) w = s[0];
        else w = word{s[0], s[1]};
        if constexpr (kNt) __builtin_nontemporal_store(w, row(tau, 0));
        else *row(tau, 0) = w;
    }
    static __device__ __forceinline__ void unpack(word w, float (&s)[V::n]) {
        if constexpr (V::n == 1) s[0] = w;
        else s[0] = w.x, s[1] = w.y;
    }
};

// Maps s -> A s + H of a thread's channels.
template <int N> struct Map {
    float A[N], H[N];
};
template <int N> __device__ __forceinline__ void compose_after(Map<N> &later, const float (&A)[N], const float (&H)[N]) {
#pragma unroll
    for (int v = 0; v < N; ++v) {   // later o (A, H)
        later.H[v] = __builtin_fmaf(later.A[v], H[v], later.H[v]);
        later.A[v] *= A[v];
    }
}

// Joins the runs of a block (step 2 above).  run: this thread's map.  Returns the state before its run in
// s_in; carry[parity] holds the state before the block, carry[parity ^ 1] receives the one after it.  One barrier
// a block suffices: arrays of one parity are written again only two barriers later.
template <typename V, int LC, int NW> struct Join {
    static constexpr int N = V::n, kSub = 64 / LC;
    float2 maps[2][NW][LC * N];
    float carry[2][LC * N];

    __device__ __forceinline__ void operator()(Map<N> run, float (&s_in)[N], float (&s_out)[N], int wave, int lane,
                                               int parity) {
        const int c = lane % LC, sub = lane / LC;
        Map<N> before;   // the runs of this wave before this one
#pragma unroll
        for (int v = 0; v < N; ++v) before.A[v] = 1.0f, before.H[v] = 0.0f;
        if constexpr (kSub > 1) {
            float A[N], H[N];
#pragma unroll
            for (int dist = LC; dist < 64; dist *= 2) {
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    A[v] = __shfl_up(run.A[v], dist);
                    H[v] = __shfl_up(run.H[v], dist);
                }
                if (lane >= dist) compose_after(run, A, H);
            }
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float a = __shfl_up(run.A[v], LC), h = __shfl_up(run.H[v], LC);
                before.A[v] = sub > 0 ? a : 1.0f;
                before.H[v] = sub > 0 ? h : 0.0f;
            }
        }
        if (sub == kSub - 1) {
#pragma unroll
            for (int v = 0; v < N; ++v) maps[parity][wave][c * N + v] = make_float2(run.A[v], run.H[v]);
        }
        __syncthreads();
        float s[N];
#pragma unroll
        for (int v = 0; v < N; ++v) s[v] = carry[parity][c * N + v];
#pragma unroll 4
        for (int w = 0; w < wave; ++w) {
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float2 m = maps[parity][w][c * N + v];
                s[v] = __builtin_fmaf(m.x, s[v], m.y);
            }
        }
#pragma unroll
        for (int v = 0; v < N; ++v) {
            s_in[v] = kSub > 1 ? __builtin_fmaf(before.A[v], s[v], before.H[v]) : s[v];
            s_out[v] = __builtin_fmaf(run.A[v], s[v], run.H[v]);
        }
        if (wave == NW - 1 && sub == kSub - 1) {
#pragma unroll
            for (int v = 0; v < N; ++v) carry[parity ^ 1][c * N + v] = s_out[v];
        }
    }
};

// Runs `count` blocks with one block of loads in flight: load(k, i) starts the loads of block i into buffer
// k, scan(k, i) works on it.  Every path to a scan has the same operations behind the loads that it waits
// for (the other buffer's loads and the stores of one block), so that the wait the compiler places there
// leaves all of them in flight; a load under a condition would make it wait for everything.
template <typename Load, typename Scan>
__device__ __forceinline__ void pipelined(int64_t count, Load load, Scan scan) {
    using B0 = IntConst<0>;
    using B1 = IntConst<1>;
    if (count <= 0) return;
    load(B0{}, 0);
    if (count == 1) {
        scan(B0{}, 0);
        return;
    }
    auto step = [&](auto next, auto current, int64_t i) {   // block i, with the loads of block i + 1 on their way
        load(next, i + 1);
        __builtin_amdgcn_sched_barrier(0);
        scan(current, i);
        __builtin_amdgcn_sched_barrier(0);
    };
    step(B1{}, B0{}, 0);
    for (int64_t i = 1;; i += 2) {
        if (i + 1 >= count) {
            scan(B1{}, i);
            return;
        }
        step(B0{}, B1{}, i);
        if (i + 2 >= count) {
            scan(B0{}, i + 1);
            return;
        }
        step(B1{}, B0{}, i + 1);
    }
}

// Work-group id -> (sequence, segment, strip).  Neighbouring strips share 128-byte lines when they are narrow, so
// consecutive strips go to work-groups of one XCD (ids 8 apart).
struct Where {
    int64_t b;
    int seg, strip;
};
__device__ __forceinline__ Where where(int strips, int n_seg) {
    const uint32_t n = gridDim.x, per = n / 8, id = blockIdx.x;
    const uint32_t v = id < per * 8 ? (id % 8) * per + id / 8 : id;
    const uint32_t row = v / (uint32_t)strips;
    return Where{(int64_t)(row / (uint32_t)n_seg), (int)(row % (uint32_t)n_seg), (int)(v % (uint32_t)strips)};
}

// This thread row's share of the maps before segment seg of a cut sequence, composed: the join of all shares
// carries the scan's starting state to the segment's.
template <typename V, int LC, int NW>
__device__ __forceinline__ Map<V::n> share_before(const SegSplit &sp, int64_t b, int seg, int D, int d, int run) {
    constexpr int N = V::n, kRuns = 64 / LC * NW;
    const int per = (sp.n_seg - 1 + kRuns - 1) / kRuns;
    Map<N> m;
#pragma unroll
    for (int v = 0; v < N; ++v) m.A[v] = 1.0f, m.H[v] = 0.0f;
    const float2 *p = sp.sums + b * sp.n_seg * D + d;
    const int k0 = run * per, k1 = min(k0 + per, seg);
#pragma unroll 4
    for (int k = k0; k < k1; ++k) {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const float2 s = p[(int64_t)k * D + v];
            m.H[v] = __builtin_fmaf(s.x, m.H[v], s.y);
            m.A[v] *= s.x;
        }
    }
    return m;
}

// The decay and input of one word of the scan: from (g, u) forward, from (g, dy) backward.
template <typename V, GateForm F, bool kRev>
__device__ __forceinline__ void scan_terms(typename V::word gw, typename V::word xw, Gate (&k)[V::n], float (&x)[V::n]) {
    float g[V::n], in[V::n];
    V::unpack(gw, g);
    V::unpack(xw, in);
#pragma unroll
    for (int v = 0; v < V::n; ++v) {
        k[v] = gate<F>(g[v]);
        x[v] = kRev ? k[v].a * in[v] : gated_input<F>(k[v], in[v]);
    }
}

}  // namespace strip

// The maps of all segments but the last of a cut sequence, which must be whole.  Each thread takes one long
// run of the segment, so nothing is joined until its end.  Memory bounds it: 1 x 65536 x 1024 bf16 in 44
// us, 6.0 TB/s.  kWholeRuns: the scan starts at a whole run of TT tokens (see gated_backward_kernel).
template <typename V, GateForm F, int LC, int NW, int TT, bool kRev, bool kWholeRuns>
__global__ __launch_bounds__(NW * 64) void gated_summary_kernel(TokenRows<const typename V::store_t> g,
                                                                TokenRows<const typename V::store_t> x,
                                                                const float *s0, const int32_t *__restrict__ lengths,
                                                                SegSplit sp, int64_t L, int D, int strips) {
    using namespace strip;
    using P = Place<V, LC, NW, TT>;
    using word = typename V::word;
    constexpr int N = V::n;
    __shared__ float2 maps[P::kRuns][LC * N];
    const Where at = where(strips, sp.n_seg - 1);
    const int64_t n = tokens_of(lengths, at.b, L);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane % LC, sub = lane / LC, words = D / N;
    const int cw = at.strip * LC + c;
    const bool live = cw < words;
    if (at.seg == 0 && threadIdx.x < LC && live) {
#pragma unroll
        for (int v = 0; v < N; ++v) sp.start[at.b * D + cw * N + v] = s0 ? s0[at.b * D + cw * N + v] : 0.0f;
    }
    const int64_t tau0 = at.seg * sp.seg_len, top = kWholeRuns ? (n + TT - 1) / TT * TT : n;
    if (tau0 + sp.seg_len > top) return;   // never read: no token lies behind a segment that is not whole
    const int64_t per = sp.seg_len / P::kRuns;   // tokens per thread, a multiple of TT
    const uint32_t cl = (uint32_t)(live ? cw : words - 1);
    Stream<V, LC, TT, kRev, false> gs(g, at.b, L, sub, cl), xs(x, at.b, L, sub, cl);
    const int64_t lane_tau = tau0 + (wave * P::kSub + sub) * per;

    Map<N> run;
#pragma unroll
    for (int v = 0; v < N; ++v) run.A[v] = 1.0f, run.H[v] = 0.0f;
    // rows of a lane: runs lie `per` tokens apart here
    const int64_t step = kRev ? -1 : 1, t0 = kRev ? top - 1 - lane_tau : lane_tau;
    // the first of this run's tokens that exists (kWholeRuns: up to TT - 1 of the first run do not)
    const int first = kWholeRuns && lane_tau == 0 ? (int)(top - n) : 0;
    const char *gp = gs.base + t0 * gs.ld + gs.chan_off, *xp = xs.base + t0 * xs.ld + xs.chan_off;
    word gw[TT], xw[TT], gn[TT], xn[TT];
    auto load = [&](word(&gd)[TT], word(&xd)[TT], int64_t i0) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            gd[i] = *reinterpret_cast<const word *>(gp + (i0 + i) * step * gs.ld);
            xd[i] = *reinterpret_cast<const word *>(xp + (i0 + i) * step * xs.ld);
        }
    };
    auto walk = [&](const word(&gd)[TT], const word(&xd)[TT], auto is_first) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            Gate k[N];
            float in[N];
            scan_terms<V, F, kRev>(gd[i], xd[i], k, in);
            const bool on = !decltype(is_first)::value || i >= first;
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float a = on ? k[v].a : 1.0f, x = on ? in[v] : 0.0f;
                run.H[v] = gated_advance(run.H[v], a, x);
                run.A[v] *= a;
            }
        }
    };
    int64_t i0 = 0;
    if constexpr (kWholeRuns) {   // the first block by itself, its positions without a token taken at the first one
        word gf[TT], xf[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int64_t r = max(i, first);
            gf[i] = *reinterpret_cast<const word *>(gp + r * step * gs.ld);
            xf[i] = *reinterpret_cast<const word *>(xp + r * step * xs.ld);
        }
        i0 = TT;
        if (i0 < per) load(gw, xw, i0);
        walk(gf, xf, std::true_type{});
    } else {
        load(gw, xw, 0);
    }
    for (; i0 < per; i0 += TT) {
        load(gn, xn, i0 + TT < per ? i0 + TT : i0);
        walk(gw, xw, std::false_type{});
#pragma unroll
        for (int i = 0; i < TT; ++i) gw[i] = gn[i], xw[i] = xn[i];
    }
#pragma unroll
    for (int v = 0; v < N; ++v) maps[wave * P::kSub + sub][c * N + v] = make_float2(run.A[v], run.H[v]);
    __syncthreads();
    for (int i = threadIdx.x; i < LC * N; i += NW * 64) {
        float A = 1.0f, H = 0.0f;
#pragma unroll 8
        for (int r = 0; r < P::kRuns; ++r) {
            const float2 m = maps[r][i];
            H = __builtin_fmaf(m.x, H, m.y);
            A *= m.x;
        }
        const int d = at.strip * LC * N + i;
        if (d < D) sp.sums[(at.b * sp.n_seg + at.seg) * D + d] = make_float2(A, H);
    }
}

// Forward scan of a strip.  Memory bounds it: 16 x 4096 x 8192 bf16 sigmoid in 587 us, 5.5 TB/s, with the
// traffic of the algorithm (2.15 GB read, 1.07 GB written); 1 x 65536 x 1024 in 32 segments in 73 us behind
// their maps, 5.5 TB/s.  Few strips leave one chain a CU: 3 x 6225 x 3864 decay with states 119 us, 4.2 TB/s.
// kSave: the state before each thread's run is kept for the backward pass, 0.5 bytes an element beside 6 (8 x 4096 x
// 8192 336 us, without 308); four waves a SIMD are asked for, which the kernels of 64 lanes have without it (else
// 140 VGPRs, one work-group a CU).
template <typename V, GateForm F, int LC, int NW, int TT, bool kNt, bool kSave>
__global__ __launch_bounds__(NW * 64, kSave && LC == 64 ? 4 : 1) void gated_scan_kernel(
    TokenRows<const typename V::store_t> g, TokenRows<const typename V::store_t> u, const float *h0,
    const int32_t *__restrict__ lengths, TokenRows<typename V::store_t> y, float *h_final, float *states, SegSplit sp,
    int64_t L, int D, int strips) {
    using namespace strip;
    using P = Place<V, LC, NW, TT>;
    using word = typename V::word;
    constexpr int N = V::n;
    __shared__ Join<V, LC, NW> join;
    const Where at = where(strips, sp.n_seg);
    const int64_t n = tokens_of(lengths, at.b, L);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane % LC, sub = lane / LC, words = D / N;
    const int cw = at.strip * LC + c;
    const uint32_t cl = (uint32_t)min(cw, words - 1);   // lanes behind the last channel repeat it, bit for bit
    const int64_t seg0 = at.seg * sp.seg_len, seg_end = min(seg0 + sp.seg_len, L);
    const int64_t end = min(seg_end, n);   // tokens [seg0, end) are scanned, [max(seg0, n), seg_end) cleared
    Stream<V, LC, TT, false, kNt> gs(g, at.b, L, sub, cl), us(u, at.b, L, sub, cl), ys(y, at.b, L, sub, cl);
    const Starts<V, LC, TT, false, kNt> starts(states, at.b, L, D, sub, cl);

    // the segment's starting state; the segment with the last token (the first one of an empty sequence) ends with
    // the final state
    float s_end[N];
#pragma unroll
    for (int v = 0; v < N; ++v) s_end[v] = 0.0f;
    const bool writes_final = seg0 < n ? seg_end >= n : (n == 0 && at.seg == 0);
    const float *begin = sp.n_seg > 1 ? sp.start : h0;
    if (wave == NW - 1 || threadIdx.x < LC) {
#pragma unroll
        for (int v = 0; v < N; ++v) s_end[v] = begin ? begin[at.b * D + (int)cl * N + v] : 0.0f;
        if (threadIdx.x < LC) {
#pragma unroll
            for (int v = 0; v < N; ++v) join.carry[at.seg > 0][c * N + v] = s_end[v];
        }
    }
    if (at.seg > 0 && seg0 < end) {
        float unused[N];
        join(share_before<V, LC, NW>(sp, at.b, at.seg, D, (int)cl * N, wave * P::kSub + sub), unused, s_end, wave,
             lane, 1);
    }

    const int64_t wave_run = (int64_t)wave * P::kSub * TT, lane_run = wave_run + sub * TT;
    struct Block {
        word g[TT], u[TT];
    } blocks[2];
    auto load = [&](Block &w, int64_t t) {   // the whole block at token t
        gs.load(w.g, t + wave_run, n, 0);
        us.load(w.u, t + wave_run, n, 0);
    };
    auto scan_block = [&](const Block &w, int64_t t, int parity, auto is_whole) {
        constexpr bool whole = decltype(is_whole)::value;
        float A[TT][N], H[TT][N];
        Map<N> run;
#pragma unroll
        for (int v = 0; v < N; ++v) run.A[v] = 1.0f, run.H[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            Gate k[N];
            float in[N];
            scan_terms<V, F, false>(w.g[i], w.u[i], k, in);
            const bool on = whole || t + lane_run + i < end;
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float a = on ? k[v].a : 1.0f, x = on ? in[v] : 0.0f;
                run.H[v] = gated_advance(run.H[v], a, x);
                run.A[v] *= a;
                A[i][v] = run.A[v];
                H[i][v] = run.H[v];
            }
        }
        float s_in[N];
        join(run, s_in, s_end, wave, lane, parity);
        if constexpr (kSave)
            if (whole || t + lane_run < end) starts.store(s_in, t + wave_run);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            float s[N];
#pragma unroll
            for (int v = 0; v < N; ++v) s[v] = __builtin_fmaf(A[i][v], s_in[v], H[i][v]);
            if (whole) {
                ys.store(V::pack(s), t + wave_run, n, i);
            } else if (t + lane_run + i < end) {
                ys.store_at(V::pack(s), t + lane_run + i);
            }
        }
    };
    const int64_t blocks_n = end > seg0 ? (end - seg0) / P::kBlock : 0, tail = seg0 + blocks_n * P::kBlock;
    pipelined(blocks_n, [&](auto k, int64_t i) { load(blocks[decltype(k)::value], seg0 + i * P::kBlock); },
              [&](auto k, int64_t i) {
                  scan_block(blocks[decltype(k)::value], seg0 + i * P::kBlock, decltype(k)::value, std::true_type{});
              });
    if (tail < end) {
        Block &w = blocks[0];
        if (tail + wave_run < end) {   // waves behind the end have nothing to load
            gs.load_clamped(w.g, tail + lane_run, n, 0, 0, n - 1);
            us.load_clamped(w.u, tail + lane_run, n, 0, 0, n - 1);
        }
        scan_block(w, tail, (int)(blocks_n & 1), std::false_type{});
    }
    if (writes_final && wave == NW - 1 && sub == P::kSub - 1) {
#pragma unroll
        for (int v = 0; v < N; ++v) h_final[at.b * D + (int)cl * N + v] = s_end[v];
    }
    const float zero[N] = {};
    for (int64_t t = max(seg0, n) + wave * P::kSub + sub; t < seg_end; t += P::kRuns) ys.store_at(V::pack(zero), t);
}

// Backward pass of a strip: the scan of c from the last token down, then the gradients of each token from c
// of the token after it and h of the token before it.  Memory bounds it: 8 x 4096 x 8192 bf16
// decay in 521 us, 5.2 TB/s; 16 x 4096 x 8192 sigmoid (six tensors) in 1156 us, 5.6 TB/s.
// Without kSaved h is read from y, which holds it in the tensors' type.  With it (y and h0 are not read) a
// thread walks its run up from the saved fp32 state, so h is in fp32 throughout; for that its runs
// have to be those of the forward scan, so scan positions count from the end of the last of them, `top`:
// up to TT - 1 positions before the last token hold none and pass c on.
// States against y: 8 x 4096 x 8192 decay 530 and 522 us, sigmoid 549 and 629 us (five tensors in place of six).
template <typename V, GateForm F, int LC, int NW, int TT, bool kNt, bool kSaved>
__global__ __launch_bounds__(NW * 64) void gated_backward_kernel(
    TokenRows<const typename V::store_t> g, TokenRows<const typename V::store_t> u,
    TokenRows<const typename V::store_t> y, TokenRows<const typename V::store_t> dy, const float *__restrict__ h0,
    const float *__restrict__ states, const float *dh_final, const int32_t *__restrict__ lengths,
    TokenRows<typename V::store_t> dg, TokenRows<typename V::store_t> du, float *dh0, SegSplit sp, int64_t L, int D,
    int strips) {
    using namespace strip;
    using P = Place<V, LC, NW, TT>;
    using word = typename V::word;
    constexpr int N = V::n;
    constexpr bool kSig = F == GateForm::Sigmoid, kReadsU = kSig || kSaved;
    __shared__ Join<V, LC, NW> join;
    const Where at = where(strips, sp.n_seg);
    const int64_t n = tokens_of(lengths, at.b, L);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane % LC, sub = lane / LC, words = D / N;
    const int cw = at.strip * LC + c;
    const uint32_t cl = (uint32_t)min(cw, words - 1);   // lanes behind the last channel repeat it, bit for bit
    // tau counts tokens from the sequence's last one (its last run's end); padding is cleared by token index
    const int64_t top = kSaved ? (n + TT - 1) / TT * TT : n, none = top - n;
    const int64_t seg0 = at.seg * sp.seg_len, seg_end = min(seg0 + sp.seg_len, L);
    const int64_t end = sp.n_seg > 1 ? min(seg0 + sp.seg_len, top) : top;
    Stream<V, LC, TT, true, kNt> gs(g, at.b, L, sub, cl), us(kReadsU ? u : g, at.b, L, sub, cl),
        hs(kSaved ? g : y, at.b, L, sub, cl), ds(dy, at.b, L, sub, cl), dgs(dg, at.b, L, sub, cl), dus(du, at.b, L, sub, cl);
    const Starts<V, LC, TT, true, kNt> starts(const_cast<float *>(states), at.b, L, D, sub, cl);

    float s_end[N];
#pragma unroll
    for (int v = 0; v < N; ++v) s_end[v] = 0.0f;
    const bool writes_final = seg0 < n ? end == top : (n == 0 && at.seg == 0);
    // a first block with positions that hold no token goes by itself, before the whole ones
    const bool head = kSaved && none > 0 && at.seg == 0 && end >= P::kBlock;
    const float *begin = sp.n_seg > 1 ? sp.start : dh_final;
    if (wave == NW - 1 || threadIdx.x < LC) {
#pragma unroll
        for (int v = 0; v < N; ++v) s_end[v] = begin ? begin[at.b * D + (int)cl * N + v] : 0.0f;
        if (threadIdx.x < LC) {
#pragma unroll
            for (int v = 0; v < N; ++v) join.carry[at.seg > 0 || head][c * N + v] = s_end[v];
        }
    }
    if (at.seg > 0 && seg0 < end) {
        float unused[N];
        join(share_before<V, LC, NW>(sp, at.b, at.seg, D, (int)cl * N, wave * P::kSub + sub), unused, s_end, wave,
             lane, 1);
    }

    const int64_t wave_run = (int64_t)wave * P::kSub * TT, lane_run = wave_run + sub * TT;
    struct Block {
        word g[TT], d[TT], h[kSaved ? 1 : TT], u[kReadsU ? TT : 1];
        float start[N];
    } blocks[2];
    auto load = [&](Block &w, int64_t tau) {   // the whole block at tau
        gs.load(w.g, tau + wave_run, top, 0);
        ds.load(w.d, tau + wave_run, top, 0);
        if constexpr (kSaved) starts.load(w.start, tau + wave_run, top);
        else hs.load(w.h, tau + wave_run, top, -1);
        if constexpr (kReadsU) us.load(w.u, tau + wave_run, top, 0);
    };
    auto load_part = [&](Block &w, int64_t tau) {   // a block with positions that hold no token, or with token 0
        if (tau + wave_run < end) {
            gs.load_clamped(w.g, tau + lane_run, top, 0, 0, n - 1);
            ds.load_clamped(w.d, tau + lane_run, top, 0, 0, n - 1);
            if constexpr (kSaved) starts.load_clamped(w.start, tau + lane_run, top);
            else hs.load_clamped(w.h, tau + lane_run, top, -1, 0, n - 1);
            if constexpr (kReadsU) us.load_clamped(w.u, tau + lane_run, top, 0, 0, n - 1);
        }
    };
    auto scan_block = [&](const Block &w, int64_t tau, int parity, auto is_whole) {
        constexpr bool whole = decltype(is_whole)::value;
        float A[TT][N], H[TT][N], b[TT][N];
        float of_c[TT][N];   // kSaved: dg = of_c c
        Map<N> run;
#pragma unroll
        for (int v = 0; v < N; ++v) run.A[v] = 1.0f, run.H[v] = 0.0f;
        auto is_on = [&](int i) {   // whether position i of this thread's run holds a token of the segment
            const int64_t at_tau = tau + lane_run + i;
            return whole || (at_tau < end && (!kSaved || at_tau >= none));
        };
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            Gate k[N];
            float in[N];
            scan_terms<V, F, true>(w.g[i], w.d[i], k, in);
            const bool on = is_on(i);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float a = on ? k[v].a : 1.0f, x = on ? in[v] : 0.0f;
                run.H[v] = gated_advance(run.H[v], a, x);
                run.A[v] *= a;
                A[i][v] = run.A[v];
                H[i][v] = run.H[v];
                if constexpr (kSig) b[i][v] = k[v].b;
            }
        }
        if constexpr (kSaved) {   // up the run from its saved state
            float h[N];
#pragma unroll
            for (int v = 0; v < N; ++v) h[v] = w.start[v];
#pragma unroll
            for (int i = TT - 1; i >= 0; --i) {
                Gate k[N];
                float in[N], uu[N];
                scan_terms<V, F, false>(w.g[i], w.u[i], k, in);
                V::unpack(w.u[i], uu);
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    of_c[i][v] = kSig ? k[v].b * (h[v] - uu[v]) : h[v];
                    h[v] = gated_advance(h[v], k[v].a, in[v]);
                }
            }
        }
        float s_in[N];
        join(run, s_in, s_end, wave, lane, parity);
        float after[N];   // c of the token after this one
#pragma unroll
        for (int v = 0; v < N; ++v) after[v] = s_in[v];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            float h[N], d[N], uu[N], out_g[N], out_u[N];
            V::unpack(w.d[i], d);
            const int64_t t = top - 1 - (tau + lane_run + i);
            if constexpr (!kSaved) {
                V::unpack(w.h[i], h);
                if constexpr (kSig) V::unpack(w.u[i], uu);
                if (!whole && t == 0) {
#pragma unroll
                    for (int v = 0; v < N; ++v) h[v] = h0 ? h0[at.b * D + (int)cl * N + v] : 0.0f;
                }
            }
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float cc = __builtin_fmaf(A[i][v], s_in[v], H[i][v]), G = d[v] + after[v];
                after[v] = cc;
                out_u[v] = kSig ? b[i][v] * G : G;
                if constexpr (kSaved) out_g[v] = cc * of_c[i][v];
                else if constexpr (kSig) out_g[v] = cc * b[i][v] * (h[v] - uu[v]);
                else out_g[v] = cc * h[v];
            }
            if (whole) {
                dgs.store(V::pack(out_g), tau + wave_run, top, i);
                dus.store(V::pack(out_u), tau + wave_run, top, i);
            } else if (is_on(i)) {
                dgs.store_at(V::pack(out_g), t);
                dus.store_at(V::pack(out_u), t);
            }
        }
    };
    // A block is whole when all its tokens (from y: and the one before each) exist.
    const int64_t begin0 = seg0 + (head ? P::kBlock : 0);
    int64_t blocks_n = end > begin0 ? (end - begin0) / P::kBlock : 0;
    if (!kSaved && blocks_n > 0 && begin0 + blocks_n * P::kBlock == n) --blocks_n;
    const int64_t tail = begin0 + blocks_n * P::kBlock;
    if constexpr (kSaved) {
        if (head) {
            load_part(blocks[0], seg0);
            scan_block(blocks[0], seg0, 1, std::false_type{});
        }
    }
    pipelined(blocks_n, [&](auto k, int64_t i) { load(blocks[decltype(k)::value], begin0 + i * P::kBlock); },
              [&](auto k, int64_t i) {
                  scan_block(blocks[decltype(k)::value], begin0 + i * P::kBlock, decltype(k)::value, std::true_type{});
              });
    if (tail < end) {
        load_part(blocks[0], tail);
        scan_block(blocks[0], tail, (int)(blocks_n & 1), std::false_type{});
    }
    if (writes_final && dh0 && wave == NW - 1 && sub == P::kSub - 1) {
#pragma unroll
        for (int v = 0; v < N; ++v) dh0[at.b * D + (int)cl * N + v] = s_end[v];
    }
    const float zero[N] = {};
    for (int64_t t = max(seg0, n) + wave * P::kSub + sub; t < seg_end; t += P::kRuns) {
        dgs.store_at(V::pack(zero), t);
        dus.store_at(V::pack(zero), t);
    }
}

// One decode token, the state in place: kVec channels of one sequence per thread, in accesses of up to 16
// bytes where all rows start on kVec elements (14 bytes an element of bf16, 8 of them the state).  256 x
// 8192 bf16 in 5.1 us, 5.8 TB/s; one sequence is a launch's latency, 2.3 us.
template <typename E, GateForm F, int kVec>
__global__ __launch_bounds__(256) void gated_step_kernel(float *__restrict__ h,
                                                         const typename E::store_t *__restrict__ g,
                                                         const typename E::store_t *__restrict__ u,
                                                         typename E::store_t *__restrict__ y, int D, int blocks_per_row,
                                                         int64_t ld_g, int64_t ld_u, int64_t ld_y) {
    using T = typename E::store_t;
    struct alignas(sizeof(T) * kVec) Values {
        T v[kVec];
    };
    struct alignas(kVec < 4 ? 4 * kVec : 16) States {
        float v[kVec];
    };
    const int64_t b = blockIdx.x / blocks_per_row;
    const int d = ((int)(blockIdx.x % blocks_per_row) * 256 + threadIdx.x) * kVec;
    if (d >= D) return;
    const Values gv = *reinterpret_cast<const Values *>(g + b * ld_g + d);
    const Values uv = *reinterpret_cast<const Values *>(u + b * ld_u + d);
    States *hp = reinterpret_cast<States *>(h + b * D + d);
    States hv = *hp;
    Values yv;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const Gate k = gate<F>(E::load(&gv.v[i]));
        hv.v[i] = gated_advance(hv.v[i], k.a, gated_input<F>(k, E::load(&uv.v[i])));
        E::store(&yv.v[i], hv.v[i]);
    }
    *hp = hv;
    *reinterpret_cast<Values *>(y + b * ld_y + d) = yv;
}

}  // namespace jscan

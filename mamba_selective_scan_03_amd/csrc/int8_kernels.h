// int8_kernels.h - a linear layer in 8-bit integers: activations quantised row by row (token by
// token), weights held as int8 with a scale for each output channel, products summed in int32.
//
//     s[m] = max(max_k |x[m][k]| * (1 / 127), 2^-126),   q[m][k] = rint(x[m][k] * (1 / s[m]))
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
// The scale of a row whose largest magnitude is amax, 1 / 127 rounded to fp32 first.  The lower bound keeps
// 1 / s finite; a row of zeros takes it and quantises to zeros.
__device__ __forceinline__ float row_scale(float amax) { return fmaxf(amax * (1.0f / 127.0f), 0x1.0p-126f); }

// Largest magnitude over a work-group of `kWaves` waves; +inf where any value is a NaN or an infinity
// (poison: the sum of the values with zero weights, 0 for finite ones).
template <int kWaves> __device__ __forceinline__ float group_amax(float amax, float poison, float *part) {
    amax = poison == 0.0f ? amax : __builtin_inff();
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    if constexpr (kWaves > 1) {
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) amax = fmaxf(amax, part[i]);
    }
    return amax;
}

// 16 bytes of x as fp32 values, and their quantised bytes.
template <typename E> struct Chunk;
template <> struct Chunk<BF16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(u32x4_t w, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <> struct Chunk<F32> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(u32x4_t w, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
};
__device__ __forceinline__ uint32_t pack4(const float *v, float r) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)__builtin_rintf(v[i] * r) & 0xffu) << (8 * i);
    return w;
}
}  // namespace quant

// Rows that start on 16 bytes, at most 64 kWaves kChunks chunks of 16 bytes long: a row stays in the registers of
// kWaves waves between its maximum and its quantisation, so x is read once.  Memory bounds it (3 bytes
// an element of bf16): 65536 x 8192 bf16 in 242 us, 6.7 TB/s.
template <typename E, int kWaves, int kChunks>
__global__ __launch_bounds__(kWaves * 64) void quantize_rows_kernel(const typename E::store_t *__restrict__ x,
                                                                    int8_t *__restrict__ q, float *__restrict__ scale,
                                                                    int64_t M, int K, int64_t ld_x) {
    using C = quant::Chunk<E>;
    __shared__ float part[kWaves];
    const int64_t m = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (m >= M) return;
    const int chunks = K / C::n;
    const u32x4_t *row = reinterpret_cast<const u32x4_t *>(x + m * ld_x);
    u32x4_t w[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int c = j * (kWaves * 64) + threadIdx.x;
        w[j] = __builtin_nontemporal_load(row + min(c, chunks - 1));   // repeats change no maximum
    }
    float amax = 0.0f, poison = 0.0f;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        float v[C::n];
        C::unpack(w[j], v);
#pragma unroll
        for (int i = 0; i < C::n; ++i) {
            amax = fmaxf(amax, fabsf(v[i]));
            poison = __builtin_fmaf(v[i], 0.0f, poison);
        }
    }
    amax = quant::group_amax<kWaves>(amax, poison, part);
    const bool finite = amax < __builtin_inff();
    const float s = finite ? quant::row_scale(amax) : __builtin_nanf(""), r = 1.0f / s;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int c = j * (kWaves * 64) + threadIdx.x;
        if (c < chunks) {
            float v[C::n];
            C::unpack(w[j], v);
            uint32_t *dst = reinterpret_cast<uint32_t *>(q + m * K + (int64_t)c * C::n);
#pragma unroll
            for (int i = 0; i < C::n / 4; ++i) dst[i] = finite ? quant::pack4(v + 4 * i, r) : 0u;
        }
    }
    if (threadIdx.x == 0) scale[m] = s;
}

// Any other row, read twice (the second time from the caches): in chunks of 16 bytes where rows start on them
// (kChunked), else element by element.
template <typename E, int kWaves, bool kChunked>
__global__ __launch_bounds__(kWaves * 64) void quantize_any_rows_kernel(const typename E::store_t *__restrict__ x,
                                                                 int8_t *__restrict__ q, float *__restrict__ scale,
                                                                 int64_t M, int K, int64_t ld_x) {
    using C = quant::Chunk<E>;
    constexpr int n = kChunked ? C::n : 1;
    __shared__ float part[kWaves];
    const int64_t m = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (m >= M) return;
    const typename E::store_t *row = x + m * ld_x;
    auto load = [&](int k, float (&v)[n]) {
        if constexpr (kChunked) C::unpack(*reinterpret_cast<const u32x4_t *>(row + k), v);
        else v[0] = E::load(row + k);
    };
    float amax = 0.0f, poison = 0.0f;
    for (int k = threadIdx.x * n; k < K; k += kWaves * 64 * n) {
        float v[n];
        load(k, v);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            amax = fmaxf(amax, fabsf(v[i]));
            poison = __builtin_fmaf(v[i], 0.0f, poison);
        }
    }
    amax = quant::group_amax<kWaves>(amax, poison, part);
    const bool finite = amax < __builtin_inff();
    const float s = finite ? quant::row_scale(amax) : __builtin_nanf(""), r = 1.0f / s;
    for (int k = threadIdx.x * n; k < K; k += kWaves * 64 * n) {
        float v[n];
        load(k, v);
        if constexpr (kChunked) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(q + m * K + k);
#pragma unroll
            for (int i = 0; i < n / 4; ++i) dst[i] = finite ? quant::pack4(v + 4 * i, r) : 0u;
        } else {
            q[m * K + k] = finite ? (int8_t)__builtin_rintf(v[0] * r) : (int8_t)0;
        }
    }
    if (threadIdx.x == 0) scale[m] = s;
}

// Four consecutive results to LDS.
template <typename E> struct Results;
template <> struct Results<BF16> {
    static __device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
};
template <> struct Results<F32> {
    static __device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};

// The output scales and biases of `kN` consecutive columns from n (those beyond N read its last one).
template <int kN> struct Columns {
    float scale[kN], bias[kN];
    __device__ __forceinline__ Columns(const float *sw, const float *b, int64_t n, int64_t N) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t c = min(n + i, N - 1);
            scale[i] = sw[c];
            bias[i] = b ? b[c] : 0.0f;
        }
    }
    // a sum as the result: scaled in fp32, the bias added (an absent one leaves the value as it is, -0 apart)
    __device__ __forceinline__ float operator()(int sum, float sq, int i) const {
        return (float)sum * sq * scale[i] + bias[i];
    }
};

// 16 rows of kCols results from LDS (rows kRow bytes apart) to rows m0 .. and columns n0 .. of the output, a P at a
// time, consecutive lanes to consecutive places.
template <typename T, typename P, int kCols, int kRow>
__device__ __forceinline__ void store_rows(T *out, const int8_t *lds, int l, int64_t m0, int64_t n0, int64_t M, int64_t N,
                                           int64_t ld_out) {
    constexpr int kPer = (int)(sizeof(P) / sizeof(T)), kPieces = kCols / kPer;
    // the narrow stores are not unrolled: their many addresses would take the registers that keep two
    // work-groups on a CU (65536 x 288 x 8192: 264 us against 186 us)
    constexpr int kUnroll = sizeof(P) == 16 ? (16 * kPieces + 63) / 64 : 1;
#pragma unroll kUnroll
    for (int j = 0; j < (16 * kPieces + 63) / 64; ++j) {
        const int c = l + 64 * j, row = c / kPieces, at = c % kPieces * kPer;
        if (16 * kPieces % 64 != 0 && c >= 16 * kPieces) break;
        const int64_t m = m0 + row, n = n0 + at;
        if (m < M && n < N) {
            const T *src = reinterpret_cast<const T *>(lds + row * kRow) + at;
            T *dst = out + m * ld_out + n;
            if (kPer == 1 || n + kPer <= N) {
                *reinterpret_cast<P *>(dst) = *reinterpret_cast<const P *>(src);
            } else {
                for (int i = 0; i < kPer && n + i < N; ++i) dst[i] = src[i];
            }
        }
    }
}

// ---- the product --------------------------------------------------------------------------------
// w is the row operand and q the column operand, so a lane's four sums of a 16 x 16 tile are four columns n of one
// output row m.  The rows of w that a wave's NT tiles hold are dealt out so that a lane's 4 NT columns are
// consecutive: result row r of tile t is column (r / 4) * 4 NT + 4 t + r % 4.
template <int NT> __device__ __forceinline__ int w_row(int t, int r) { return (r >> 2) * 4 * NT + 4 * t + (r & 3); }

// A BM x BN tile per work-group, K in stages of 128 bytes.  WR x WC waves make the tile; with KG > 1 as
// many groups of waves take every KG-th stage each and add their sums through LDS at the end, which
// shortens the chain of stages where tiles are too few to fill the chip. 16384 x 16384 x 4096 with 256 x
// 256 tiles in 0.95 ms, 2.3 POP/s: the power limit holds the clock at about 1.6 GHz, and the matrix cores
// are busy for 57 to 60% of it.  1 x 16384 x 4096 in 17.6 us with w read from memory, 3.8 TB/s (11.9 us from the
// last-level cache).  77 x 4096 x 8192 in 14.5 us (13.0): the latency of the stages.  A stage's rows of q and w
// go from memory straight into LDS, kBufs - 1 stages (one to three) ahead of the products.  A row's eight 16-byte
// chunks are permuted by (row / 2) % 8, so that the 16 rows of one operand read fall on distinct banks.
namespace tiled {
constexpr int kStage = 128;
constexpr int kGroup = 8;   // tile rows that are walked together, column by column, so that tiles in
                            // flight on one XCD share their rows of q and w in its L2
}  // namespace tiled

// 16 bytes per lane from base + off straight into LDS at lds + 16 * lane (see lds_dma16), the uniform base in
// scalar registers.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma16_at(const void *base, uint32_t off, uint32_t lds) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)b) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(u), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// A work-group barrier that leaves loads into LDS in flight (__syncthreads() waits for all of them); its release
// fence waits for the wave's earlier LDS reads.
__device__ __forceinline__ void block_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// s_waitcnt operand that leaves n vector-memory operations in flight (gfx9: bits 0-3 and 14-15 of the
// count; the expcnt and lgkmcnt fields at their maxima do not wait).
template <int n> constexpr int vmcnt_at_most() { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// waves per SIMD of the work-groups that LDS lets onto a CU
constexpr int waves_per_simd(int waves, int lds_bytes) {
    const int n = 163840 / lds_bytes * waves / 4;
    return n < 1 ? 1 : n > 8 ? 8 : n;
}

template <typename E, int BM, int BN, int WR, int WC, int KG, int kBufs>
__global__ __launch_bounds__(KG * WR * WC * 64,
                             waves_per_simd(KG * WR * WC, KG * kBufs * (BM + BN) * 128)) void matmul_i8_tiled_kernel(
    const int8_t *__restrict__ q, const float *__restrict__ sq, const int8_t *__restrict__ w,
    const float *__restrict__ sw, const float *__restrict__ bias, typename E::store_t *__restrict__ out, int64_t M,
    int64_t N, int64_t K, int64_t ld_out, int m_tiles, int n_tiles, int wide) {
    using namespace tiled;
    constexpr int MT = BM / WR / 16, NT = BN / WC / 16, kWaves = WR * WC;
    // DMA instructions of a stage (8 rows each), dealt out to the waves in turn
    constexpr int kInst = (BM + BN) / 8, kPer = (kInst + kWaves - 1) / kWaves;
    static_assert(BM % 8 == 0 && BN % 8 == 0, "stages are whole wave instructions");
    static_assert(kBufs == 2 || kInst % kWaves == 0, "with more buffers a wave counts its loads in flight");
    __shared__ __attribute__((aligned(16))) int8_t stages_of[KG][kBufs][(BM + BN) * kStage];

    // tile of this work-group: consecutive tiles to one XCD (ids 8 apart)
    const uint32_t total = gridDim.x, per = total / 8, id = blockIdx.x;
    const uint32_t v = id < per * 8 ? (id % 8) * per + id / 8 : id;
    const uint32_t group = v / (kGroup * n_tiles), in = v % (kGroup * n_tiles);
    const uint32_t rows_here = min((uint32_t)kGroup, (uint32_t)m_tiles - group * kGroup);
    const int64_t m0 = (int64_t)(group * kGroup + in % rows_here) * BM, n0 = (int64_t)(in / rows_here) * BN;

    const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, r16 = l & 15, g4 = l >> 4;
    const int wave = wave_id % kWaves, kg = wave_id / kWaves, wr = wave / WC, wc = wave % WC;
    int8_t(*stage)[(BM + BN) * kStage] = stages_of[kg];

    // This wave's DMA instructions fill LDS rows 8 (wave + kWaves j) ..; LDS rows 0 .. BM - 1 are q's, then w's in
    // tile order.  Offsets from the tile's first row; rows beyond the matrix re-read its last one.
    // The chunk that lane l brings to its place: (row / 2) % 8 of row 8 i + l / 8 is l / 16 + 4 (i % 2).
    auto chunk = [&](int j) { return (l & 7) ^ (l >> 4) ^ (((wave + kWaves * j) & 1) << 2); };
    uint32_t off[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int row = 8 * (wave + kWaves * j) + (l >> 3);
        int64_t r;
        if (row < BM) {
            r = min((int64_t)row, M - 1 - m0);
        } else {
            const int s = row - BM, strip = s / (16 * NT), t = s % (16 * NT) / 16;
            r = min((int64_t)(strip * 16 * NT + w_row<NT>(t, s % 16)), N - 1 - n0);
        }
        off[j] = (uint32_t)(r * K) + 16 * chunk(j);
    }
    const int8_t *qb = q + m0 * K, *wb = w + n0 * K;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)&stages_of[0][0][0] +
                          kg * kBufs * ((BM + BN) * kStage);
    auto dma = [&](int64_t k0, int buf) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int first = 8 * (wave + kWaves * j);
            if (kInst % kWaves != 0 && first >= BM + BN) continue;
            // chunks behind the end of a row re-read its last one; the products leave them out
            const int over = max((int)(k0 - (K - 16)) + 16 * chunk(j), 0);
            lds_dma16_at((first < BM ? qb : wb) + k0, off[j] - (uint32_t)over,
                         lds0 + buf * ((BM + BN) * kStage) + first * kStage);
        }
    };

    i32x4_t acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] = i32x4_t{0, 0, 0, 0};

    auto operand = [&](const int8_t *s, int row, int k) {
        return *reinterpret_cast<const i32x4_t *>(s + row * kStage + 16 * ((4 * k + g4) ^ ((row >> 1) & 7)));
    };
    const int64_t stages = (K + kStage - 1) / kStage, rounds = (stages + KG - 1) / KG;
#pragma unroll
    for (int i = 0; i < kBufs - 1; ++i)
        if (i * KG + kg < stages) dma((i * KG + kg) * kStage, i);
    int buf = 0;
    for (int64_t round = 0; round < rounds; ++round) {
        const int64_t st = round * KG + kg;
        // this wave's loads of the stage have landed; those of the kBufs - 2 stages behind it may be in flight
        if (kBufs > 2 && st + (kBufs - 2) * KG < stages) __builtin_amdgcn_s_waitcnt(vmcnt_at_most<(kBufs - 2) * kPer>());
        else __builtin_amdgcn_s_waitcnt(vmcnt_at_most<0>());
        block_barrier();   // every wave's part is in; every wave is done with the stage before
        const int next = buf == 0 ? kBufs - 1 : buf - 1;   // the buffer of the stage before
        if (st + (kBufs - 1) * KG < stages) dma((st + (kBufs - 1) * KG) * kStage, next);
        if (KG > 1 && st >= stages) break;   // the last round, where no barrier follows in the loop
        const int8_t *s = stage[buf];
        buf = buf == kBufs - 1 ? 0 : buf + 1;
        const int64_t left = K - st * kStage;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            i32x4_t a[MT], b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) b[t] = operand(s, BM + wc * 16 * NT + 16 * t + r16, k);
#pragma unroll
            for (int u = 0; u < MT; ++u) a[u] = operand(s, wr * 16 * MT + 16 * u + r16, k);
            if (left < kStage) {   // chunks behind the end of the rows
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (16 * (4 * k + g4) >= left) b[t] = i32x4_t{0, 0, 0, 0};
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < MT; ++u) acc[t][u] = mfma_i8(b[t], a[u], acc[t][u]);
        }
    }

    // Results go out through LDS, 16 rows of a wave at a time, so that a store covers whole rows of the
    // wave's columns (straight from the registers a store touches 64 pieces of 8 bytes: 16384 x 16384 x
    // 256 took 762 us).
    using T = typename E::store_t;
    constexpr int kCols = 16 * NT;
    constexpr int kRow = kCols * (int)sizeof(T) + 16;   // bytes, padded off the banks' period
    static_assert(kWaves * 16 * kRow <= (int)sizeof(stages_of), "the results fit the stages");
    __syncthreads();   // every wave is done with the operands
    if constexpr (KG > 1) {   // the groups' sums to group 0, which goes on alone
        i32x4_t *sums = reinterpret_cast<i32x4_t *>(&stages_of[0][0][0]);
        constexpr int kTile = NT * MT * 64;   // a wave's sums
        static_assert((KG - 1) * kWaves * kTile * 16 <= (int)sizeof(stages_of), "the groups' sums fit the stages");
        if (kg > 0) {
            i32x4_t *to = sums + ((kg - 1) * kWaves + wave) * kTile + l;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < MT; ++u) to[(t * MT + u) * 64] = acc[t][u];
        }
        __syncthreads();
        if (kg == 0) {
#pragma unroll
            for (int k = 0; k < KG - 1; ++k) {
                const i32x4_t *from = sums + (k * kWaves + wave) * kTile + l;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < MT; ++u) acc[t][u] += from[(t * MT + u) * 64];
            }
        }
        __syncthreads();
        if (kg > 0) return;
    }
    int8_t *mine = &stages_of[0][0][0] + wave * 16 * kRow;
    const int64_t nw = n0 + wc * kCols;
    const Columns<4 * NT> col(sw, bias, min(nw + g4 * 4 * NT, N - 1), N);
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int64_t mu = m0 + wr * 16 * MT + 16 * u;
        const float s = sq[min(mu + r16, M - 1)];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = col(acc[t][u][i], s, 4 * t + i);
            Results<E>::store4(reinterpret_cast<T *>(mine + r16 * kRow) + g4 * 4 * NT + 4 * t, v);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (wide == 16) store_rows<T, u32x4_t, kCols, kRow>(out, mine, l, mu, nw, M, N, ld_out);
        else if (wide == 4) store_rows<T, uint32_t, kCols, kRow>(out, mine, l, mu, nw, M, N, ld_out);
        else store_rows<T, T, kCols, kRow>(out, mine, l, mu, nw, M, N, ld_out);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

}  // namespace jscan

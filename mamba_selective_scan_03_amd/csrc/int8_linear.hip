// int8_linear.hip - host entry points of the int8 projection (include/jscan.h): the row quantiser and
// the product with int8 weights.
#include "host_common.h"
#include "int8_kernels.h"

using namespace jscan::host;

namespace {

constexpr int64_t kMaxK = 131056;   // 128 * 128 * K stays below 2^31

bool dims_ok(int64_t M, int64_t K) {
    return M >= 0 && M <= ((int64_t)1 << 30) && K >= 0 && K % 16 == 0 && K <= kMaxK;
}

// Rows on 16 bytes stay in registers: one wave for short ones, four up to 1024 chunks of 16 bytes (8192 bf16
// values), sixteen up to 4096; the rest is read twice.
template <typename E>
void launch_quantize(const void *x, int8_t *q, float *scale, int64_t M, int64_t K, int64_t ld_x, hipStream_t s) {
    const auto *xt = static_cast<const typename E::store_t *>(x);
    const int64_t per = 16 / (int64_t)sizeof(typename E::store_t), chunks = K / per;
    // rows over both dimensions: one dimension counts 2^32 work-items
    const int64_t across = M < (1 << 20) ? M : (1 << 20);
    const dim3 grid((unsigned)across, (unsigned)((M + across - 1) / across));
    auto launch = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, grid, dim3((unsigned)threads), 0, s, xt, q, scale, M, (int)K, ld_x);
    };
    const bool on16 = aligned16(x) && ld_x % per == 0;
    if (!on16 && K <= 8192) launch(jscan::quantize_any_rows_kernel<E, 4, false>, 256);
    else if (!on16) launch(jscan::quantize_any_rows_kernel<E, 16, false>, 1024);
    else if (chunks > 4096) launch(jscan::quantize_any_rows_kernel<E, 16, true>, 1024);
    else if (chunks <= 128) launch(jscan::quantize_rows_kernel<E, 1, 2>, 64);
    else if (chunks <= 512) launch(jscan::quantize_rows_kernel<E, 4, 2>, 256);
    else if (chunks <= 1024) launch(jscan::quantize_rows_kernel<E, 4, 4>, 256);
    else launch(jscan::quantize_rows_kernel<E, 16, 4>, 1024);
}

// The tiles of the product and what they take on this chip (us, bf16 output; fitted to 710 products of random sizes
// up to 16384, times in profiles/sweep_int8_tiles.txt): `start` of a work-group, `round` from one of its stages to the
// next, `stage` of a CU's work for one stage of one tile, with `per_cu` work-groups side by side on a CU.
struct Tile {
    int bm, bn, groups, threads, per_cu;
    float start, round, stage;
};
constexpr Tile kTiles[] = {
    {16, 16, 8, 512, 1, 0.95f, 0.40f, 0.057f},   {16, 32, 4, 512, 2, 1.1f, 0.19f, 0.083f},
    {32, 32, 4, 512, 1, 1.2f, 0.50f, 0.12f},     {64, 32, 4, 512, 1, 1.75f, 0.48f, 0.177f},
    {64, 64, 2, 512, 1, 1.65f, 0.53f, 0.26f},    {64, 64, 1, 256, 3, 1.45f, 0.285f, 0.265f},
    {64, 128, 1, 256, 2, 2.35f, 0.39f, 0.424f},  {128, 128, 1, 512, 2, 2.5f, 0.72f, 0.61f},
    {128, 144, 1, 256, 2, 5.2f, 0.60f, 0.70f},   {256, 256, 1, 1024, 1, 6.7f, 1.41f, 1.41f}};
constexpr float kLaunch = 2.0f;

int64_t tiles_of(const Tile &t, int64_t M, int64_t N) { return ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn); }

// The tile that is expected to take least: large ones read least per product, small ones fill the chip when
// rows and columns are few, K dealt out to groups of waves shortens the chain of stages, and the 144 columns leave
// less of a tile empty for some widths.  A CU runs its share of the tiles per_cu at a time; each turn
// costs a start, and all of them the larger of the time along the stages and the time of the CU's work.
// Measured with w read from memory (M x N x K):
//     1 x 4096 x 8192: 16 x 16 tiles 8.9 us, 16 x 32 10.0, 64 x 64 25
//     77 x 4096 x 8192: 64 x 32 13.7 us, 32 x 32 20, 64 x 64 25 (in two groups 18.5)
//     256 x 4096 x 8192: 64 x 64 in two groups 20.9 us, in one 26, 64 x 32 28
//     512 x 4096 x 8192: 64 x 128 32 us, 64 x 64 35 (in two groups 38), 128 x 128 55
//     512 x 16384 x 4096: 128 x 128 41 us, 256 x 256 54, 64 x 128 57
//     2048 x 8192 x 4096: 256 x 256 58 us, 128 x 128 73
//     65536 x 288 x 8192: 128 x 144 183 us, 128 x 128 228, 256 x 256 219
// Over products of random sizes the choice is 1 to 2% slower than the best of these and six other tiles.  Only tiles
// whose launch one dimension can count (all but for enormous outputs); -1 where there is none.
int choose_tile(int64_t M, int64_t N, int64_t K) {
    const int64_t stages = (K + 127) / 128;
    int best = -1;
    float least = 0.0f;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        const Tile &t = kTiles[i];
        const int64_t tiles = tiles_of(t, M, N);
        if (tiles > kMaxItems / t.threads) continue;
        const float share = (float)((tiles + 255) / 256), turns = (float)(((tiles + 255) / 256 + t.per_cu - 1) / t.per_cu);
        const float along = turns * (float)((stages + t.groups - 1) / t.groups) * t.round;
        const float work = share * (float)stages * t.stage;
        const float us = kLaunch + turns * t.start + (along > work ? along : work);
        if (best < 0 || us < least) best = i, least = us;
    }
    return best;
}

struct MatmulArgs {
    const int8_t *q;
    const float *sq;
    const int8_t *w;
    const float *sw, *bias;
    void *out;
    int64_t M, N, K, ld_out;
    hipStream_t stream;
};

template <typename E, int BM, int BN, int WR, int WC, int KG, int kBufs> void launch_tiled(const MatmulArgs &a) {
    using T = typename E::store_t;
    const int m_tiles = (int)((a.M + BM - 1) / BM), n_tiles = (int)((a.N + BN - 1) / BN);
    // the widest store that every output row starts on
    const uint64_t start = reinterpret_cast<uint64_t>(a.out) | (uint64_t)(a.ld_out * (int64_t)sizeof(T));
    const int wide = start % 16 == 0 ? 16 : start % 4 == 0 ? 4 : 2;
    hipLaunchKernelGGL((jscan::matmul_i8_tiled_kernel<E, BM, BN, WR, WC, KG, kBufs>),
                       dim3((unsigned)((int64_t)m_tiles * n_tiles)), dim3(KG * WR * WC * 64), 0, a.stream, a.q, a.sq,
                       a.w, a.sw, a.bias, static_cast<T *>(a.out), a.M, a.N, a.K, a.ld_out, m_tiles, n_tiles, wide);
}

template <typename E> void launch_matmul(const MatmulArgs &a) {
    switch (choose_tile(a.M, a.N, a.K)) {
    case 0: launch_tiled<E, 16, 16, 1, 1, 8, 3>(a); break;
    case 1: launch_tiled<E, 16, 32, 1, 2, 4, 3>(a); break;
    case 2: launch_tiled<E, 32, 32, 2, 1, 4, 4>(a); break;
    case 3: launch_tiled<E, 64, 32, 2, 1, 4, 3>(a); break;
    case 4: launch_tiled<E, 64, 64, 2, 2, 2, 3>(a); break;
    case 5: launch_tiled<E, 64, 64, 2, 2, 1, 3>(a); break;
    case 6: launch_tiled<E, 64, 128, 2, 2, 1, 3>(a); break;
    case 7: launch_tiled<E, 128, 128, 2, 4, 1, 2>(a); break;
    case 8: launch_tiled<E, 128, 144, 4, 1, 1, 2>(a); break;
    default: launch_tiled<E, 256, 256, 4, 4, 1, 2>(a); break;
    }
}

}  // namespace

extern "C" {

jscan_status jscan_quantize_rows(const void *x, int8_t *q, float *scale, int64_t M, int64_t K, int64_t ld_x,
                                 jscan_dtype dtype, void *stream) {
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!dims_ok(M, K) || K == 0) return JSCAN_ERR_SHAPE;
    if (M == 0) return JSCAN_OK;
    if (ld_x < K || ld_x > ((int64_t)1 << 58) / M) return JSCAN_ERR_SHAPE;
    if (!x || !q || !scale) return JSCAN_ERR_NULL;
    const int64_t es = elem_bytes(dtype);
    if (!aligned(x, es) || !aligned16(q) || !aligned(scale, 4)) return JSCAN_ERR_ALIGN;
    const Span sx = span(Rows{x, M, K * es, ld_x * es}), sq = span(q, M * K), ss = span(scale, M * 4);
    if (overlaps(sx, sq) || overlaps(sx, ss) || overlaps(sq, ss)) return JSCAN_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == JSCAN_BF16) launch_quantize<jscan::BF16>(x, q, scale, M, K, ld_x, s);
    else launch_quantize<jscan::F32>(x, q, scale, M, K, ld_x, s);
    return launch_status();
}

jscan_status jscan_matmul_i8(const int8_t *q, const float *q_scale, const int8_t *w, const float *w_scale,
                             const float *bias, void *out, int64_t M, int64_t N, int64_t K, int64_t ld_out,
                             jscan_dtype dtype, void *stream) {
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!dims_ok(M, K) || K == 0 || N < 0 || N > (1 << 24))
        return JSCAN_ERR_SHAPE;
    if (M == 0 || N == 0) return JSCAN_OK;
    if (choose_tile(M, N, K) < 0) return JSCAN_ERR_SHAPE;
    if (ld_out < N || ld_out > ((int64_t)1 << 58) / M) return JSCAN_ERR_SHAPE;
    if (!q || !q_scale || !w || !w_scale || !out) return JSCAN_ERR_NULL;
    const int64_t es = elem_bytes(dtype);
    if (!aligned16(q) || !aligned16(w) || !aligned(out, es) || !aligned(q_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(bias, 4))
        return JSCAN_ERR_ALIGN;
    const Span so = span(Rows{out, M, N * es, ld_out * es});
    const Span in[] = {span(q, M * K), span(q_scale, M * 4), span(w, N * K), span(w_scale, N * 4),
                       span(bias, bias ? N * 4 : 0)};
    for (const Span &i : in)
        if (overlaps(so, i)) return JSCAN_ERR_ALIAS;
    const MatmulArgs a{q, q_scale, w, w_scale, bias, out, M, N, K, ld_out, static_cast<hipStream_t>(stream)};
    if (dtype == JSCAN_BF16) launch_matmul<jscan::BF16>(a);
    else launch_matmul<jscan::F32>(a);
    return launch_status();
}

}  // extern "C"

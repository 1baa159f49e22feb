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
    if (dtype == JSCAN_BF16)
        hipLaunchKernelGGL(jscan::quantize_rows_kernel<jscan::BF16>, dim3((unsigned)M), dim3(jscan::quant::kThreads), 0,
                           s, static_cast<const uint16_t *>(x), q, scale, K, ld_x);
    else
        hipLaunchKernelGGL(jscan::quantize_rows_kernel<jscan::F32>, dim3((unsigned)M), dim3(jscan::quant::kThreads), 0,
                           s, static_cast<const float *>(x), q, scale, K, ld_x);
    return launch_status();
}

jscan_status jscan_matmul_i8(const int8_t *q, const float *q_scale, const int8_t *w, const float *w_scale,
                             const float *bias, void *out, int64_t M, int64_t N, int64_t K, int64_t ld_out,
                             jscan_dtype dtype, void *stream) {
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!dims_ok(M, K) || K == 0 || N < 0 || N > (1 << 24) || ((M + 15) / 16) * ((N + 15) / 16) > kMaxBlocks)
        return JSCAN_ERR_SHAPE;
    if (M == 0 || N == 0) return JSCAN_OK;
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
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t m_tiles = (M + 15) / 16, n_tiles = (N + 15) / 16;
    const dim3 grid((unsigned)(m_tiles * n_tiles));
    if (dtype == JSCAN_BF16)
        hipLaunchKernelGGL(jscan::matmul_i8_kernel<jscan::BF16>, grid, dim3(64), 0, s, q, q_scale, w, w_scale, bias,
                           static_cast<uint16_t *>(out), M, N, K, ld_out, (int)n_tiles);
    else
        hipLaunchKernelGGL(jscan::matmul_i8_kernel<jscan::F32>, grid, dim3(64), 0, s, q, q_scale, w, w_scale, bias,
                           static_cast<float *>(out), M, N, K, ld_out, (int)n_tiles);
    return launch_status();
}

}  // extern "C"

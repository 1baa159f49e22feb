// norm.hip - host entry points of the root-mean-square norm (include/jscan.h): with the residual's addition, into the
// tensor's type or into 8 bits, and its backward pass.
#include "host_common.h"
#include "norm_kernels.h"

using namespace jscan::host;
using jscan::NormRows;

namespace {

constexpr int64_t kMostRows = (int64_t)1 << 30, kMostK = (int64_t)1 << 24, kMostInt8K = 131056;

// A row's pieces over waves: one wave for short rows, four up to 1024 pieces of 16 bytes, sixteen up to 4096; no
// more pieces a thread than that takes.  Rows shorter than a piece and longer ones go element by element.
struct Layout {
    int waves, chunks;   // chunks 0: element by element
};
Layout layout_for(int64_t K, int64_t es) {
    const int64_t n = 16 / es, pieces = (K + n - 1) / n;
    if (K < n) return {1, 0};
    if (pieces > 4096) return {16, 0};
    const int waves = pieces <= 128 ? 1 : pieces <= 1024 ? 4 : 16;
    return {waves, (int)((pieces + waves * 64 - 1) / (waves * 64))};
}

constexpr int64_t kMostGroups = (int64_t)1 << 20;   // of a launch

// Work-groups of the forward call: a row each, more only beyond the largest launch.
int64_t forward_groups(int64_t M) { return M < kMostGroups ? M : kMostGroups; }

// Work-groups of the backward pass, each of which goes on to further rows and leaves a share of the gain's gradient; one
// for a row, or for a few short ones, which writes that gradient itself and spares the launch that adds the shares, about
// 4 us of the host's time.  On the GPU (us, one work-group and one a row with that launch; bf16): 8 x 64 5.5 and 4.6, 8 x
// 2048 6.9 and 5.8, 4 x 4096 5.9 and 6.5, 2 x 8192 5.8 and 6.8; beyond the limit 8 x 4096 9.1 and 6.5, 8 x 16384 21 and
// 9.7, 2 x 32768 37 and 29, 8 x 65536 271 and 41.
constexpr int64_t kFewRows = 8, kFewValues = 16384;
int64_t backward_groups(const Layout &l, int64_t M, int64_t K) {
    if (M <= 1 || (M <= kFewRows && M * K <= kFewValues)) return M > 0 ? 1 : 0;
    const int64_t each = l.chunks == 0 ? 1 : jscan::norm::rows_at_once(l.waves, l.chunks);
    const int64_t most = l.waves == 1 ? 1024 : l.waves == 4 ? 512 : 256;   // four, eight, sixteen waves a CU
    const int64_t rows = (M + each - 1) / each;
    return rows < most ? rows : most;
}

// Tensors beyond the last-level cache go by with the non-temporal hint.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

struct NormArgs {
    Pair x, residual, y, total, dy, dtotal, dx;
    const float *gain;
    int8_t *q;
    float *scale, *partial;
    int64_t M, K, groups;
    float eps;
    hipStream_t stream;
};

template <typename T> NormRows<const T> in_rows(Pair t) { return {static_cast<const T *>(t.p), t.ld}; }
template <typename T> NormRows<T> out_rows(Pair t) { return {static_cast<T *>(const_cast<void *>(t.p)), t.ld}; }

template <typename E, int kWaves, int kChunks, bool kInt8> void launch_forward(const NormArgs &a) {
    constexpr int64_t kEach = (int64_t)sizeof(typename E::store_t);
    using T = typename E::store_t;
    const jscan::NormOut<E> out{out_rows<T>(a.y), a.q, a.scale};
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)a.groups), dim3(kWaves * 64), 0, a.stream, in_rows<T>(a.x),
                           in_rows<T>(a.residual), a.gain, out, out_rows<T>(a.total), a.M, (int)a.K, a.eps);
    };
    if constexpr (kChunks == 0) launch(jscan::rms_norm_any_kernel<E, kWaves, kInt8>);
    else if (a.residual.p && a.M * a.K * kEach * 4 > kStreamBytes)
        launch(jscan::rms_norm_kernel<E, kWaves, kChunks, kInt8, true, true>);
    else if (a.residual.p) launch(jscan::rms_norm_kernel<E, kWaves, kChunks, kInt8, true, false>);
    else if (a.M * a.K * kEach * 2 > kStreamBytes)
        launch(jscan::rms_norm_kernel<E, kWaves, kChunks, kInt8, false, true>);
    else launch(jscan::rms_norm_kernel<E, kWaves, kChunks, kInt8, false, false>);
}

template <typename E, int kWaves, int kChunks> void launch_backward(const NormArgs &a) {
    const bool streams = a.M * a.K * (int64_t)sizeof(typename E::store_t) * 4 > kStreamBytes;
    using T = typename E::store_t;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)a.groups), dim3(kWaves * 64), 0, a.stream, in_rows<T>(a.total), a.gain,
                           in_rows<T>(a.dy), in_rows<T>(a.dtotal), out_rows<T>(a.dx), a.partial, a.M, (int)a.K, a.eps);
    };
    if constexpr (kChunks == 0) launch(jscan::rms_norm_backward_any_kernel<E, kWaves>);
    else if (a.dtotal.p && streams) launch(jscan::rms_norm_backward_kernel<E, kWaves, kChunks, true, true>);
    else if (a.dtotal.p) launch(jscan::rms_norm_backward_kernel<E, kWaves, kChunks, true, false>);
    else if (streams) launch(jscan::rms_norm_backward_kernel<E, kWaves, kChunks, false, true>);
    else launch(jscan::rms_norm_backward_kernel<E, kWaves, kChunks, false, false>);
}

// Calls f<waves, chunks>() for a layout.
template <typename F> void with_layout(const Layout &l, F f) {
    using jscan::IntConst;
    auto two_or_more = [&](auto w) {
        if (l.chunks == 2) f(w, IntConst<2>{});
        else if (l.chunks == 3) f(w, IntConst<3>{});
        else f(w, IntConst<4>{});
    };
    if (l.chunks == 0) {
        if (l.waves == 1) f(IntConst<1>{}, IntConst<0>{});
        else f(IntConst<16>{}, IntConst<0>{});
    } else if (l.waves == 1) {
        if (l.chunks == 1) f(IntConst<1>{}, IntConst<1>{});
        else f(IntConst<1>{}, IntConst<2>{});
    } else if (l.waves == 4) {
        if (l.chunks == 1) f(IntConst<4>{}, IntConst<1>{});
        else two_or_more(IntConst<4>{});
    } else {
        two_or_more(IntConst<16>{});
    }
}

template <bool kInt8> void run_forward(NormArgs &a, jscan_dtype dtype) {
    const Layout l = layout_for(a.K, elem_bytes(dtype));
    a.groups = forward_groups(a.M);
    with_layout(l, [&](auto w, auto c) {
        if (dtype == JSCAN_BF16) launch_forward<jscan::BF16, decltype(w)::value, decltype(c)::value, kInt8>(a);
        else launch_forward<jscan::F32, decltype(w)::value, decltype(c)::value, kInt8>(a);
    });
}

bool sizes_ok(int64_t M, int64_t K, float eps) { return M >= 0 && M <= kMostRows && K >= 1 && K <= kMostK && eps >= 0.0f; }

// The checks of x, residual, gain and total that both forward calls share; total may be x or residual itself.
jscan_status check_inputs(Pair x, Pair residual, const float *gain, Pair total, int64_t M, int64_t K, int64_t es) {
    if (!ld_ok(x.ld, M, K) || (residual.p && !ld_ok(residual.ld, M, K)) || (total.p && !ld_ok(total.ld, M, K)))
        return JSCAN_ERR_SHAPE;
    if (!x.p || !gain || (total.p && !residual.p)) return JSCAN_ERR_NULL;
    if (!aligned(x.p, es) || !aligned(residual.p, es) || !aligned(total.p, es) || !aligned(gain, 4)) return JSCAN_ERR_ALIGN;
    auto is = [&](Pair t) { return total.p && t.p == total.p && (t.ld == total.ld || M == 1); };
    const Rows out[] = {rows_of(total, M, K, es)};
    const Rows in[] = {rows_of(is(x) ? Pair{nullptr, 0} : x, M, K, es), rows_of(is(residual) ? Pair{nullptr, 0} : residual, M, K, es),
                       flat(gain, K * 4)};
    return any_overlap(out, in) ? JSCAN_ERR_ALIAS : JSCAN_OK;
}

}  // namespace

extern "C" {

jscan_status jscan_rms_norm(const void *x, const void *residual, const float *gain, void *y, void *total, int64_t M,
                            int64_t K, int64_t ld_x, int64_t ld_residual, int64_t ld_y, int64_t ld_total, float eps,
                            jscan_dtype dtype, void *stream) {
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!sizes_ok(M, K, eps)) return JSCAN_ERR_SHAPE;
    if (M == 0) return JSCAN_OK;
    const int64_t es = elem_bytes(dtype);
    if (!ld_ok(ld_y, M, K)) return JSCAN_ERR_SHAPE;
    if (!y) return JSCAN_ERR_NULL;
    if (!aligned(y, es)) return JSCAN_ERR_ALIGN;
    NormArgs a{};
    a.x = {x, ld_x}, a.residual = {residual, ld_residual}, a.y = {y, ld_y}, a.total = {total, ld_total};
    const jscan_status st = check_inputs(a.x, a.residual, gain, a.total, M, K, es);
    if (st != JSCAN_OK) return st;
    const Rows out[] = {rows_of(a.y, M, K, es)};
    const Rows in[] = {rows_of(a.x, M, K, es), rows_of(a.residual, M, K, es), flat(gain, K * 4), rows_of(a.total, M, K, es)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    a.gain = gain, a.M = M, a.K = K, a.eps = eps, a.stream = static_cast<hipStream_t>(stream);
    run_forward<false>(a, dtype);
    return launch_status();
}

jscan_status jscan_rms_norm_quantize(const void *x, const void *residual, const float *gain, int8_t *q, float *scale,
                                     void *total, int64_t M, int64_t K, int64_t ld_x, int64_t ld_residual,
                                     int64_t ld_total, float eps, jscan_dtype dtype, void *stream) {
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!sizes_ok(M, K, eps) || K % 16 != 0 || K > kMostInt8K) return JSCAN_ERR_SHAPE;
    if (M == 0) return JSCAN_OK;
    const int64_t es = elem_bytes(dtype);
    if (!q || !scale) return JSCAN_ERR_NULL;
    if (!aligned16(q) || !aligned(scale, 4)) return JSCAN_ERR_ALIGN;
    NormArgs a{};
    a.x = {x, ld_x}, a.residual = {residual, ld_residual}, a.total = {total, ld_total};
    const jscan_status st = check_inputs(a.x, a.residual, gain, a.total, M, K, es);
    if (st != JSCAN_OK) return st;
    const Rows out[] = {flat(q, M * K), flat(scale, M * 4)};
    const Rows in[] = {rows_of(a.x, M, K, es), rows_of(a.residual, M, K, es), flat(gain, K * 4), rows_of(a.total, M, K, es)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    a.gain = gain, a.q = q, a.scale = scale, a.M = M, a.K = K, a.eps = eps, a.stream = static_cast<hipStream_t>(stream);
    run_forward<true>(a, dtype);
    return launch_status();
}

// Room for the groups of either type: rows of fp32 take four waves where those of bf16 take one.
int64_t jscan_rms_norm_backward_workspace(int64_t M, int64_t K) {
    if (!sizes_ok(M, K, 0.0f)) return -1;
    const int64_t a = backward_groups(layout_for(K, 2), M, K), b = backward_groups(layout_for(K, 4), M, K);
    const int64_t groups = a > b ? a : b;
    return groups <= 1 ? 0 : groups * K * 4;
}

jscan_status jscan_rms_norm_backward(const void *total, const float *gain, const void *dy, const void *dtotal, void *dx,
                                     float *dgain, int64_t M, int64_t K, int64_t ld_total, int64_t ld_dy,
                                     int64_t ld_dtotal, int64_t ld_dx, void *workspace, int64_t workspace_bytes, float eps,
                                     jscan_dtype dtype, void *stream) {
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!sizes_ok(M, K, eps)) return JSCAN_ERR_SHAPE;
    if (M > 0 && (!ld_ok(ld_total, M, K) || !ld_ok(ld_dy, M, K) || !ld_ok(ld_dx, M, K) || (dtotal && !ld_ok(ld_dtotal, M, K))))
        return JSCAN_ERR_SHAPE;
    if (!gain || !dgain || (M > 0 && (!total || !dy || !dx))) return JSCAN_ERR_NULL;
    if (M == 0) total = dy = dtotal = dx = nullptr;
    const int64_t es = elem_bytes(dtype), need = jscan_rms_norm_backward_workspace(M, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return JSCAN_ERR_WORKSPACE;
    if (!aligned(total, es) || !aligned(dy, es) || !aligned(dtotal, es) || !aligned(dx, es) || !aligned(gain, 4) ||
        !aligned(dgain, 4) || (need > 0 && !aligned16(workspace)))
        return JSCAN_ERR_ALIGN;
    NormArgs a{};
    a.total = {total, ld_total}, a.dy = {dy, ld_dy}, a.dtotal = {dtotal, ld_dtotal}, a.dx = {dx, ld_dx};
    const bool same = dx && dx == dtotal && (ld_dx == ld_dtotal || M == 1);
    const Rows out[] = {rows_of(a.dx, M, K, es), flat(dgain, K * 4), flat(workspace, need)};
    const Rows in[] = {rows_of(a.total, M, K, es), rows_of(a.dy, M, K, es), flat(gain, K * 4),
                       rows_of(same ? Pair{nullptr, 0} : a.dtotal, M, K, es)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    a.gain = gain, a.partial = static_cast<float *>(workspace), a.M = M, a.K = K, a.eps = eps;
    a.stream = static_cast<hipStream_t>(stream);
    if (M > 0) {
        const Layout l = layout_for(K, es);
        a.groups = backward_groups(l, M, K);
        if (a.groups == 1) a.partial = dgain;
        with_layout(l, [&](auto w, auto c) {
            if (dtype == JSCAN_BF16) launch_backward<jscan::BF16, decltype(w)::value, decltype(c)::value>(a);
            else launch_backward<jscan::F32, decltype(w)::value, decltype(c)::value>(a);
        });
        if (launch_status() != JSCAN_OK) return JSCAN_ERR_HIP;
        if (a.groups == 1) return JSCAN_OK;
    }
    hipLaunchKernelGGL(jscan::norm_gain_kernel, dim3((unsigned)((K + 63) / 64)), dim3(1024), 0, a.stream, a.partial, dgain,
                       a.groups, (int)K);
    return launch_status();
}

}  // extern "C"

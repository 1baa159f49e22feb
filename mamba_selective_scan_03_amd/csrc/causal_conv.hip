// causal_conv.hip - host entry points of the short causal convolution (include/jscan.h): whole sequences, the
// backward pass and the decode step.
#include "causal_conv_kernels.h"
#include "host_common.h"

using namespace jscan::host;
using jscan::Act;
using jscan::TokenRows;

namespace {

constexpr int64_t kMostGroups = (int64_t)1 << 23;   // work-groups of one launch

bool width_ok(int64_t W) { return W >= 2 && W <= 4; }
bool activation_ok(jscan_activation a) { return a == JSCAN_ACT_NONE || a == JSCAN_ACT_SILU; }

// Channels a thread takes: four, where a row has them; two in the backward pass of tensors that do not stream (us for four
// with 1024 waves and two with 2048: 24 x 1000 x 500 bf16 27 and 24, 5 x 1001 x 1000 fp32 21 and 19, 1 x 16384 x 2048
// bf16 53 and 50; 1 x 32768 x 2048, which streams, 82 and 103).
int channels_of(int64_t D) { return D < 4 ? 1 : 4; }
int backward_channels_of(int64_t D, bool streamed) { return D < 2 ? 1 : streamed ? 4 : 2; }

// As long a run as leaves `least` waves, from 8 tokens to `most`; longer ones only where a launch could not count the
// work-groups of one sequence.
jscan::conv::Split split_for(int64_t batch, int64_t L, int64_t D, int n, int64_t least, int64_t most) {
    const int64_t words = (D + n - 1) / n;
    int log = 0;
    while (log < 6 && ((int64_t)1 << log) < words) ++log;
    const int64_t rows = jscan::conv::kThreads >> log, strips = (words + (1 << log) - 1) >> log;
    int64_t run = most;
    auto segs = [&] { return L > rows * run ? (L + rows * run - 1) / (rows * run) : 1; };
    while (run > 8 && batch * strips * segs() * (jscan::conv::kThreads / 64) < least) run /= 2;
    while (strips * segs() > kMostGroups) run *= 2;
    return {log, (int)strips, (int)segs(), run};
}

// Tensors beyond the last-level cache go by with the non-temporal hint (us, 8 x 4096 x 8192 bf16, without and with it:
// forward 204 and 192, backward 329 and 298; from the cache the loads lose by it: 24 x 1000 x 500 11.6 and 14.8).
constexpr int64_t kStreamBytes = (int64_t)256 << 20;
bool streams(int64_t batch, int64_t L, int64_t D, int64_t es, int tensors) {
    return D >= 4 && batch * L * D * es * tensors > kStreamBytes;
}

// Forward: runs of 64 tokens, 32 where the tensors stream (8 x 4096 x 8192: 204 us for 212; 1 x 32768 x 2048: 60 for 56).
// Backward: a run computes W - 1 more tokens than it has, and its shares of the taps' gradients are written once (us
// for 128 tokens, 256, 64: 8 x 4096 x 8192 329, 352, 378).
constexpr int64_t kForwardWaves = 4096, kForwardRun = 64, kForwardStreamRun = 32;
constexpr int64_t kBackwardWaves = 2048, kBackwardStreamWaves = 1024, kBackwardRun = 128;

jscan::conv::Split backward_split(int64_t batch, int64_t L, int64_t D, bool streamed) {
    return split_for(batch, L, D, backward_channels_of(D, streamed), streamed ? kBackwardStreamWaves : kBackwardWaves,
                     kBackwardRun);
}

// Room for the shares of either type: fp32 streams where bf16 does not.
int64_t backward_workspace_bytes(int64_t batch, int64_t L, int64_t D, int64_t W) {
    if (batch == 0 || D == 0) return 0;
    int64_t segs = backward_split(batch, L, D, false).segs;
    if (D >= 4) {
        const int64_t streamed = backward_split(batch, L, D, true).segs;
        if (streamed > segs) segs = streamed;
    }
    return batch * segs * (W + 1) * D * 4;
}

struct ConvArgs {
    Pair x, y, dy, dx;
    const void *state;
    const float *w, *bias;
    const int32_t *lengths;
    void *state_out;
    const void *dstate_out;
    void *dstate;
    float *partial;
    int64_t batch, L, D;
    jscan::conv::Split split;
    bool streams;
    hipStream_t stream;
};

template <typename T> TokenRows<const T> in_rows(Pair t, int64_t row) {
    return {t.p ? static_cast<const T *>(t.p) + row * t.ld : nullptr, t.ld};
}
template <typename T> TokenRows<T> out_rows(Pair t, int64_t row) {
    return {t.p ? static_cast<T *>(const_cast<void *>(t.p)) + row * t.ld : nullptr, t.ld};
}
template <typename T> T *from(const void *p, int64_t i) {
    return p ? static_cast<T *>(const_cast<void *>(p)) + i : nullptr;
}

// Launches of as many sequences as one can count.
template <typename F> void by_sequences(const ConvArgs &a, F launch) {
    const int64_t each = (int64_t)a.split.strips * a.split.segs, most = kMostGroups / each;
    for (int64_t b = 0; b < a.batch; b += most) {
        const int64_t count = most < a.batch - b ? most : a.batch - b;
        launch(b, dim3((unsigned)(count * each)));
    }
}

template <typename E, int N, int W, Act A, bool kNt> void launch_forward(const ConvArgs &a) {
    using T = typename E::store_t;
    if constexpr (N > 1 && !kNt) {
        if (a.streams) return launch_forward<E, N, W, A, true>(a);
    }
    by_sequences(a, [&](int64_t b, dim3 grid) {
        hipLaunchKernelGGL((jscan::causal_conv_kernel<E, N, W, A, kNt>), grid, dim3(jscan::conv::kThreads), 0, a.stream,
                           in_rows<T>(a.x, b * a.L), from<const T>(a.state, b * (W - 1) * a.D), a.w, a.bias,
                           from<const int32_t>(a.lengths, b), out_rows<T>(a.y, b * a.L),
                           from<T>(a.state_out, b * (W - 1) * a.D), a.L, (int)a.D, a.split);
    });
}

template <typename E, int N, int W, Act A> void launch_backward(const ConvArgs &a) {
    using T = typename E::store_t;
    constexpr bool kNt = N == 4;   // see backward_channels_of
    by_sequences(a, [&](int64_t b, dim3 grid) {
        hipLaunchKernelGGL((jscan::causal_conv_backward_kernel<E, N, W, A, kNt>), grid, dim3(jscan::conv::kThreads), 0,
                           a.stream, in_rows<T>(a.x, b * a.L), from<const T>(a.state, b * (W - 1) * a.D), a.w, a.bias,
                           from<const int32_t>(a.lengths, b), in_rows<T>(a.dy, b * a.L),
                           from<const T>(a.dstate_out, b * (W - 1) * a.D), out_rows<T>(a.dx, b * a.L),
                           from<T>(a.dstate, b * (W - 1) * a.D),
                           a.partial + b * a.split.segs * (W + 1) * a.D, a.L, (int)a.D, a.split);
    });
}

// Sequences a thread of the step takes: four where that leaves a wave for every SIMD (their taps are 40 bytes a thread, against
// 4 of each token).  It takes two channels (us for four: 256 x 8192 bf16 6.9 and 7.7, fp32 14.4 and 14.6).
constexpr int64_t kStepRows = 4, kStepWaves = 1024;

template <typename E, int N, int W, Act A, int kRows>
void launch_step(void *state, const void *x, const float *w, const float *bias, void *y, int64_t batch, int64_t D,
                 int64_t ld_x, int64_t ld_y, hipStream_t stream) {
    using T = typename E::store_t;
    const int64_t words = D / N;
    if constexpr (kRows == 1) {
        if (batch * words >= kStepRows * kStepWaves * 64)
            return launch_step<E, N, W, A, kStepRows>(state, x, w, bias, y, batch, D, ld_x, ld_y, stream);
    }
    const int64_t rows = kMostGroups * jscan::conv::kThreads / words * kRows;   // of one launch
    for (int64_t b = 0; b < batch; b += rows) {
        const int64_t count = rows < batch - b ? rows : batch - b;
        const int64_t threads = (count + kRows - 1) / kRows * words;
        hipLaunchKernelGGL((jscan::causal_conv_step_kernel<E, N, W, A, kRows>),
                           dim3((unsigned)((threads + jscan::conv::kThreads - 1) / jscan::conv::kThreads)),
                           dim3(jscan::conv::kThreads), 0, stream, static_cast<T *>(state) + b * (W - 1) * D,
                           static_cast<const T *>(x) + b * ld_x, w, bias, static_cast<T *>(y) + b * ld_y, count, (int)D,
                           (int)words, ld_x, ld_y);
    }
}

// Calls f<type, channels, width, activation>(); channels is one of Ns.
template <typename E, int N, int W, typename F> void with_activation(jscan_activation a, F f) {
    if (a == JSCAN_ACT_SILU) f(E{}, jscan::IntConst<N>{}, jscan::IntConst<W>{}, jscan::IntConst<(int)Act::Silu>{});
    else f(E{}, jscan::IntConst<N>{}, jscan::IntConst<W>{}, jscan::IntConst<(int)Act::None>{});
}
template <typename E, int N, typename F> void with_width(int64_t W, jscan_activation a, F f) {
    if (W == 2) with_activation<E, N, 2>(a, f);
    else if (W == 3) with_activation<E, N, 3>(a, f);
    else with_activation<E, N, 4>(a, f);
}
template <typename E, int... Ns, typename F> void with_channels(int n, int64_t W, jscan_activation a, F f) {
    ((n == Ns ? with_width<E, Ns>(W, a, f) : void()), ...);
}
template <int... Ns, typename F> void dispatch(jscan_dtype dtype, int n, int64_t W, jscan_activation a, F f) {
    if (dtype == JSCAN_BF16) with_channels<jscan::BF16, Ns...>(n, W, a, f);
    else with_channels<jscan::F32, Ns...>(n, W, a, f);
}

jscan_status check_kind(jscan_activation activation, jscan_dtype dtype) {
    if (!activation_ok(activation)) return JSCAN_ERR_FORM;
    return dtype == JSCAN_F32 || dtype == JSCAN_BF16 ? JSCAN_OK : JSCAN_ERR_DTYPE;
}

}  // namespace

extern "C" {

jscan_status jscan_causal_conv(const void *x, const void *state, const float *w, const float *bias,
                               const int32_t *lengths, void *y, void *state_out, int64_t batch, int64_t L, int64_t D,
                               int64_t W, int64_t ld_x, int64_t ld_y, jscan_activation activation, jscan_dtype dtype,
                               void *stream) {
    const jscan_status kind = check_kind(activation, dtype);
    if (kind != JSCAN_OK) return kind;
    if (!shape_ok(batch, L, D) || !width_ok(W)) return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) return JSCAN_OK;
    const int64_t rows = batch * L, es = elem_bytes(dtype), state_bytes = batch * (W - 1) * D * es;
    if (!ld_ok(ld_x, rows, D) || !ld_ok(ld_y, rows, D)) return JSCAN_ERR_SHAPE;
    if (!w || (L > 0 && (!x || !y))) return JSCAN_ERR_NULL;
    if (L == 0) x = y = nullptr;
    for (const void *p : {x, (const void *)y, state, (const void *)state_out})
        if (!aligned(p, es)) return JSCAN_ERR_ALIGN;
    if (!aligned(w, 4) || !aligned(bias, 4) || !aligned(lengths, 4)) return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of({y, ld_y}, rows, D, es), flat(state_out, state_bytes)};
    const Rows in[] = {rows_of({x, ld_x}, rows, D, es), flat(state == state_out ? nullptr : state, state_bytes),
                       flat(w, D * W * 4), flat(bias, D * 4), flat(lengths, batch * 4)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    // A state updated in place at a D that four does not divide: the last word of a row would read what the word before it
    // has written, so a thread takes one channel, without the non-temporal hint (us, with a state of its own for the
    // output, four channels, and in place: 16 x 4096 x 8193 bf16 501 and 536, 8 x 4096 x 8193 249 and 255, 24 x 1000 x 501
    // 11.9 both, 5 x 1001 x 1001 fp32 8.0 and 7.7).
    const int n = state && state == state_out && D % 4 != 0 ? 1 : channels_of(D);
    ConvArgs a{};
    a.x = {x, ld_x}, a.y = {y, ld_y}, a.state = state, a.state_out = state_out, a.w = w, a.bias = bias;
    a.lengths = lengths, a.batch = batch, a.L = L, a.D = D, a.stream = static_cast<hipStream_t>(stream);
    a.streams = n > 1 && streams(batch, L, D, es, 2);
    a.split = split_for(batch, L, D, n, kForwardWaves, a.streams ? kForwardStreamRun : kForwardRun);
    dispatch<4, 1>(dtype, n, W, activation, [&](auto e, auto n_c, auto w_c, auto a_c) {
        launch_forward<decltype(e), decltype(n_c)::value, decltype(w_c)::value, (Act)decltype(a_c)::value, false>(a);
    });
    return launch_status();
}

int64_t jscan_causal_conv_backward_workspace(int64_t batch, int64_t L, int64_t D, int64_t W) {
    return shape_ok(batch, L, D) && width_ok(W) ? backward_workspace_bytes(batch, L, D, W) : -1;
}

jscan_status jscan_causal_conv_backward(const void *x, const void *state, const float *w, const float *bias,
                                        const int32_t *lengths, const void *dy, const void *dstate_out, void *dx,
                                        void *dstate, float *dw, float *dbias, int64_t batch, int64_t L, int64_t D,
                                        int64_t W, int64_t ld_x, int64_t ld_dy, int64_t ld_dx, void *workspace,
                                        int64_t workspace_bytes, jscan_activation activation, jscan_dtype dtype,
                                        void *stream) {
    const jscan_status kind = check_kind(activation, dtype);
    if (kind != JSCAN_OK) return kind;
    if (!shape_ok(batch, L, D) || !width_ok(W)) return JSCAN_ERR_SHAPE;
    if (D == 0) return JSCAN_OK;
    const int64_t rows = batch * L, es = elem_bytes(dtype), state_bytes = batch * (W - 1) * D * es;
    if (!ld_ok(ld_x, rows, D) || !ld_ok(ld_dy, rows, D) || !ld_ok(ld_dx, rows, D)) return JSCAN_ERR_SHAPE;
    if (!w || !dw || (rows > 0 && (!x || !dy || !dx))) return JSCAN_ERR_NULL;
    if (rows == 0) x = dy = dx = nullptr;
    if (batch == 0) state = dstate_out = dstate = nullptr;
    const int64_t need = backward_workspace_bytes(batch, L, D, W);
    if (need > 0 && (!workspace || workspace_bytes < need)) return JSCAN_ERR_WORKSPACE;
    for (const void *p : {x, dy, (const void *)dx, state, dstate_out, (const void *)dstate})
        if (!aligned(p, es)) return JSCAN_ERR_ALIGN;
    for (const void *p : {(const void *)w, (const void *)bias, (const void *)lengths, (const void *)dw, (const void *)dbias})
        if (!aligned(p, 4)) return JSCAN_ERR_ALIGN;
    if (need > 0 && !aligned16(workspace)) return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of({dx, ld_dx}, rows, D, es), flat(dstate, state_bytes), flat(dw, D * W * 4),
                        flat(dbias, D * 4), flat(workspace, need)};
    const Rows in[] = {rows_of({x, ld_x}, rows, D, es), rows_of({dy, ld_dy}, rows, D, es), flat(state, state_bytes),
                       flat(dstate_out, state_bytes), flat(w, D * W * 4), flat(bias, D * 4), flat(lengths, batch * 4)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    ConvArgs a{};
    a.x = {x, ld_x}, a.dy = {dy, ld_dy}, a.dx = {dx, ld_dx}, a.state = state, a.dstate_out = dstate_out;
    a.dstate = dstate, a.w = w, a.bias = bias, a.lengths = lengths, a.partial = static_cast<float *>(workspace);
    a.batch = batch, a.L = L, a.D = D, a.stream = static_cast<hipStream_t>(stream);
    int64_t shares = 0;   // none without a sequence: the gradients of taps and bias are then zeros
    if (batch > 0) {
        const bool streamed = streams(batch, L, D, es, 3);
        a.split = backward_split(batch, L, D, streamed);
        shares = batch * a.split.segs;
        dispatch<4, 2, 1>(dtype, backward_channels_of(D, streamed), W, activation, [&](auto e, auto n_c, auto w_c, auto a_c) {
            launch_backward<decltype(e), decltype(n_c)::value, decltype(w_c)::value, (Act)decltype(a_c)::value>(a);
        });
        if (launch_status() != JSCAN_OK) return JSCAN_ERR_HIP;
    }
    const dim3 grid((unsigned)((D + 63) / 64), (unsigned)(W + 1));
    if (W == 2) hipLaunchKernelGGL(jscan::conv_sum_kernel<2>, grid, dim3(1024), 0, a.stream, a.partial, dw, dbias, shares, (int)D);
    else if (W == 3) hipLaunchKernelGGL(jscan::conv_sum_kernel<3>, grid, dim3(1024), 0, a.stream, a.partial, dw, dbias, shares, (int)D);
    else hipLaunchKernelGGL(jscan::conv_sum_kernel<4>, grid, dim3(1024), 0, a.stream, a.partial, dw, dbias, shares, (int)D);
    return launch_status();
}

jscan_status jscan_causal_conv_step(void *state, const void *x_t, const float *w, const float *bias, void *y_t,
                                    int64_t batch, int64_t D, int64_t W, int64_t ld_x, int64_t ld_y,
                                    jscan_activation activation, jscan_dtype dtype, void *stream) {
    const jscan_status kind = check_kind(activation, dtype);
    if (kind != JSCAN_OK) return kind;
    if (!shape_ok(batch, 1, D) || !width_ok(W)) return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) return JSCAN_OK;
    if (!ld_ok(ld_x, batch, D) || !ld_ok(ld_y, batch, D)) return JSCAN_ERR_SHAPE;
    if (!state || !x_t || !w || !y_t) return JSCAN_ERR_NULL;
    const int64_t es = elem_bytes(dtype);
    if (!aligned(state, es) || !aligned(x_t, es) || !aligned(y_t, es) || !aligned(w, 4) || !aligned(bias, 4))
        return JSCAN_ERR_ALIGN;
    const Rows out[] = {flat(state, batch * (W - 1) * D * es), rows_of({y_t, ld_y}, batch, D, es)};
    const Rows in[] = {rows_of({x_t, ld_x}, batch, D, es), flat(w, D * W * 4), flat(bias, D * 4)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    // the state is updated in place, so no two words may share a channel
    dispatch<2, 1>(dtype, D % 2 == 0 ? 2 : 1, W, activation, [&](auto e, auto n_c, auto w_c, auto a_c) {
        launch_step<decltype(e), decltype(n_c)::value, decltype(w_c)::value, (Act)decltype(a_c)::value, 1>(
            state, x_t, w, bias, y_t, batch, D, ld_x, ld_y, static_cast<hipStream_t>(stream));
    });
    return launch_status();
}

}  // extern "C"

// prefill_gate.hip - host entry points of the selective scan with its skip and output gate (include/jscan.h): whole
// sequences, token by token or time-parallel, and the decode step.  The kernels are those of the scan without
// them, instantiated with kGate: the arithmetic of the scan bounds them as it does without, and the gate adds a logistic
// function to a token's sixteen exponentials and a fourth tensor to the three.  Measured, bf16 (us, and without skip and
// gate): 1 x 65536 x 8192 token by token as the scan sums 1860 (1766), with fp32 sums (chunk 0) 2086; 1 x 65536 x 1024 in
// segments 343 (328); step 256 x 8192 46.5, 6.1 TB/s.
#include "prefill_host.h"
#include "prefill_lane_kernel.h"
#include "step_kernel.h"

using namespace jscan::host;
using jscan::AForm;
using jscan::OutGate;

namespace {

// Whether the launches of a plan can be counted.
bool gate_grids_fit(int64_t batch, int64_t D, const ChunkPlan &p) {
    const int64_t pairs = (batch * D * JSCAN_D_STATE + jscan::carry::kPairs - 1) / jscan::carry::kPairs;
    return chunk_grids_fit(batch, D, p) && batch * p.n_seg * ((D + 255) / 256) * 256 <= kMaxItems &&
           pairs * jscan::carry::kThreads <= kMaxItems;
}

constexpr int64_t kMostGateStride = (int64_t)1 << 25;   // elements between rows of z (32-bit byte offsets of 8 rows)

// How an automatic call scans: the way that is expected to take least, token by token or in segments of seg_len tokens.
// Times in us, from one GPU of 256 CUs (bf16 with fp32 sums; fp32 takes up to 1.13 times that):
//     rows kernel    a work-group a CU at a time, each 8 and 0.031 a token       (1 x 65536 x 8192 2086, 8 x 639 x 416 24)
//     lane kernel    0.65 a token for few waves, 0.58 more for a wave a SIMD     (3 x 688 x 144 453, 24 x 847 x 5704 1508)
//     segments       15, a token of both passes 0.66 to 1.25 with one to four waves a SIMD, which is what fits at a
//                    time, and 700 bytes for a channel's states and A in each,
//                    0.002 a channel more where the segments are more than 16    (1 x 65536 x 1024 in 256 345, in 512 384;
//                    1 x 3932 x 32 in 16 26, in 256 179; 1 x 8192 x 1024 in 64 73; 24 x 847 x 5704 in 384 671)
// Over 28 shapes the choice is at most 1.28 times the best segment length tried.  jscan_prefill_chunked's own rule
// (segments of 256 tokens and more wherever channels are fewer than 8192) takes 220 us for 1 x 3932 x 32, 163 for 1 x
// 8192 x 1024, and 165 for 1 x 512 x 4096, which takes 21 token by token.
ChunkPlan plan_automatic(int64_t batch, int64_t L, int64_t D) {
    const float channels = (float)batch * (float)D, tokens = (float)L;
    float least;
    if (jscan::rows_kernel_applies(batch, D)) {
        const int64_t groups = batch * (D / jscan::rows::kCh);
        least = (float)((groups + 255) / 256) * (0.031f * tokens + 8.0f);
        if (groups > 256) least *= 0.7f;   // left only for a clear gain: 13 x 95 x 5664 takes 60, in segments of 32 77
    } else {
        const float waves = (float)(batch * ((D + 63) / 64)) / 1024.0f;   // a SIMD
        const float token = 0.55f + 0.58f * waves;
        least = 8.0f + tokens * (token > 0.65f ? token : 0.65f);
    }
    ChunkPlan best;
    best.seg_len = L;
    for (const int64_t seg : {16, 32, 48, 64, 96, 128, 192, 256, 384, 512, 768, 1024, 2048, 4096}) {
        if (seg >= L) break;
        ChunkPlan p;
        p.seg_len = seg;
        p.n_seg = (L + seg - 1) / seg;
        if (!gate_grids_fit(batch, D, p)) continue;
        const float waves = (float)(batch * p.n_seg * ((D + 255) / 256)) / 256.0f;   // a SIMD
        const float token = waves <= 1.0f ? 0.66f : waves <= 2.0f ? 0.70f : 1.25f * __builtin_ceilf(waves / 4.0f);
        const float carry = p.n_seg > jscan::carry::kGroups ? 2.0e-3f * channels : 0.0f;
        const float us = 15.0f + token * (float)seg + channels * (float)p.n_seg * 700.0f / 5.0e6f + carry;
        if (us < least) least = us, best = p;
    }
    return best;
}

struct GateArgs {
    const void *x, *delta;
    const float *A;
    const void *B, *C;
    float *h;   // the step's state
    const float *h0;
    void *y;
    float *h_final;
    int64_t batch, L, D, ld_xd, ld_bc, ld_y;
    OutGate gate;
    bool fp32_sum;   // with a chunk given or 0, so that the precision does not follow the way that the shape is scanned
    hipStream_t stream;
};

template <typename T> const T *at(const void *p, int64_t i) { return p ? static_cast<const T *>(p) + i : nullptr; }

// Sequences b .. b + n - 1 of a call, for launches that one dimension can count.
template <typename E> GateArgs sequences(const GateArgs &a, int64_t b, int64_t n) {
    using T = typename E::store_t;
    GateArgs s = a;
    s.x = at<T>(a.x, b * a.L * a.D);
    s.delta = at<T>(a.delta, b * a.L * a.D);
    s.B = at<T>(a.B, b * a.L * jscan::kDState);
    s.C = at<T>(a.C, b * a.L * jscan::kDState);
    s.h0 = at<float>(a.h0, b * a.D * jscan::kDState);
    s.y = const_cast<T *>(at<T>(a.y, b * a.L * a.D));
    s.h_final = a.h_final + b * a.D * jscan::kDState;
    s.gate.z = at<T>(a.gate.z, b * a.L * a.gate.ld_z);
    s.batch = n;
    return s;
}

template <typename E, AForm AF> void launch_sequences(const GateArgs &a) {
    using T = typename E::store_t;
    const jscan::Segments sg{a.L, a.L, 1, 0};
    const T *x = static_cast<const T *>(a.x), *dl = static_cast<const T *>(a.delta);
    const T *B = static_cast<const T *>(a.B), *C = static_cast<const T *>(a.C);
    T *y = static_cast<T *>(a.y);
    if (jscan::rows_kernel_applies(a.batch, a.D)) {
        auto launch = [&](auto fp32_sum) {
            jscan::launch_prefill_rows<E, false, AF, false, true, decltype(fp32_sum)::value != 0>(
                x, dl, a.A, B, C, a.h0, y, a.h_final, sg, a.batch, (int)a.D, a.stream,
                jscan::DeltaProj{nullptr, nullptr, nullptr}, jscan::Trap{nullptr, nullptr, nullptr}, a.gate);
        };
        if constexpr (sizeof(T) == 2 && AF == AForm::Diagonal) {
            if (a.fp32_sum) return launch(jscan::IntConst<1>{});
        }
        launch(jscan::IntConst<0>{});
        return;
    }
    const int blocks = (int)((a.D + 63) / 64);
    hipLaunchKernelGGL((jscan::prefill_lane_kernel<E, AF, false, true>), dim3((unsigned)(a.batch * blocks)), dim3(64), 0,
                       a.stream, x, dl, a.A, B, C, a.h0, y, a.h_final, sg, (int)a.D, blocks,
                       jscan::Trap{nullptr, nullptr, nullptr}, a.gate);
}

template <typename E, AForm AF> void launch_prefill(const GateArgs &a) {
    const int64_t items = jscan::rows_kernel_applies(a.batch, a.D) ? a.D / jscan::rows::kCh * jscan::rows::kThreads
                                                                   : (a.D + 63) / 64 * 64;   // of a sequence
    const int64_t each = kMaxItems / items;
    for (int64_t b = 0; b < a.batch; b += each)
        launch_sequences<E, AF>(sequences<E>(a, b, each < a.batch - b ? each : a.batch - b));
}

template <typename E> jscan_status launch_chunked(const GateArgs &a, const ChunkPlan &p, void *workspace) {
    using T = typename E::store_t;
    float *hbuf = static_cast<float *>(workspace), *dsum = hbuf + a.batch * p.n_seg * a.D * jscan::kDState;
    const int64_t nrows = a.batch * p.n_seg;
    const T *x = static_cast<const T *>(a.x), *dl = static_cast<const T *>(a.delta);
    const T *B = static_cast<const T *>(a.B), *C = static_cast<const T *>(a.C);
    T *y = static_cast<T *>(a.y);
    // the passes of jscan_prefill_chunked: only the last one writes y
    const jscan::Segments each{a.L, p.seg_len, (int)p.n_seg, 0}, again{a.L, p.seg_len, (int)p.n_seg, 1};
    jscan::launch_prefill_seg_lane<E, true, true>(x, dl, a.A, B, C, nullptr, nullptr, hbuf, dsum, each, nrows, (int)a.D,
                                                  a.stream);
    if (launch_status() != JSCAN_OK) return JSCAN_ERR_HIP;
    jscan::launch_chunk_carry(hbuf, dsum, a.A, a.h0, a.batch * a.D * jscan::kDState, (int)a.D, (int)p.n_seg, a.stream);
    if (launch_status() != JSCAN_OK) return JSCAN_ERR_HIP;
    if (jscan::rows_kernel_applies(a.batch, a.D))
        jscan::launch_prefill_seg_lane<E, false, true, true>(x, dl, a.A, B, C, hbuf, y, a.h_final, nullptr, again, nrows,
                                                             (int)a.D, a.stream, a.gate);
    else
        jscan::launch_prefill_seg_lane<E, false, false, true>(x, dl, a.A, B, C, hbuf, y, a.h_final, nullptr, again, nrows,
                                                              (int)a.D, a.stream, a.gate);
    return launch_status();
}

template <typename E, AForm AF> void launch_step(const GateArgs &a) {
    using T = typename E::store_t;
    constexpr int kRows = jscan::step::kRows;
    const int blocks = (int)((a.D * 4 + 255) / 256);
    const int64_t each = kMaxItems / ((int64_t)blocks * 256) * kRows;   // rows of one launch
    for (int64_t b = 0; b < a.batch; b += each) {
        const int64_t n = each < a.batch - b ? each : a.batch - b;
        OutGate gate = a.gate;
        gate.z = at<T>(a.gate.z, b * a.gate.ld_z);
        hipLaunchKernelGGL((jscan::step_kernel<E, AF, false, true>), dim3((unsigned)((n + kRows - 1) / kRows * blocks)),
                           dim3(256), 0, a.stream, a.h + b * a.D * jscan::kDState, at<T>(a.x, b * a.ld_xd),
                           at<T>(a.delta, b * a.ld_xd), a.A, at<T>(a.B, b * a.ld_bc), at<T>(a.C, b * a.ld_bc),
                           static_cast<T *>(a.y) + b * a.ld_y, (int)n, (int)a.D, blocks, a.ld_xd, a.ld_bc, a.ld_y, nullptr,
                           nullptr, nullptr, gate);
    }
}

// Calls f with the type and the form as compile-time values.
template <typename F> void dispatch(jscan_dtype dtype, AForm af, F f) {
    auto by_form = [&](auto e) {
        if (af == AForm::ScaledIdentity) f(e, jscan::IntConst<(int)AForm::ScaledIdentity>{});
        else if (af == AForm::ComplexPairs) f(e, jscan::IntConst<(int)AForm::ComplexPairs>{});
        else f(e, jscan::IntConst<(int)AForm::Diagonal>{});
    };
    if (dtype == JSCAN_BF16) by_form(jscan::BF16{});
    else by_form(jscan::F32{});
}

// The gate's own arguments, for `rows` rows of y (y's rows are ld_y elements apart).
jscan_status check_gate(const float *skip, const void *z, int64_t ld_z, const void *y, int64_t ld_y, const float *h,
                        int64_t rows, int64_t batch, int64_t D, int64_t es) {
    if (!skip && !z) return JSCAN_ERR_NULL;
    if (z && (ld_z < D || ld_z % 8 != 0 || ld_z > kMostGateStride)) return JSCAN_ERR_SHAPE;
    if ((skip && !aligned(skip, 4)) || (z && !aligned16(z))) return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of({y, ld_y}, rows, D, es), flat(h, batch * D * JSCAN_D_STATE * 4)};
    const Rows in[] = {rows_of({z, ld_z}, rows, D, es), flat(skip, D * 4)};
    return any_overlap(out, in) ? JSCAN_ERR_ALIAS : JSCAN_OK;
}

}  // namespace

extern "C" {

int64_t jscan_prefill_gate_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t chunk) {
    if (batch < 0 || L < 0 || D < 0 || N != JSCAN_D_STATE || D % 8 != 0 || D > (1 << 24) || batch > (1 << 20) || chunk < -1)
        return -1;
    if (batch == 0 || L == 0 || D == 0 || chunk < 0) return 0;
    const ChunkPlan p = chunk > 0 ? plan_chunks(batch, L, D, chunk) : plan_automatic(batch, L, D);
    return p.n_seg > 1 && !gate_grids_fit(batch, D, p) ? -1 : chunk_workspace_bytes(p, batch, D);
}

jscan_status jscan_prefill_gate(const void *x, const void *delta, const float *A, const void *B, const void *C,
                                const float *h0, const float *skip, const void *z, void *y, float *h_final, int64_t batch,
                                int64_t L, int64_t D, int64_t N, int64_t ld_z, int64_t chunk, void *workspace,
                                int64_t workspace_bytes, jscan_a_form a_form, jscan_dtype dtype, void *stream) {
    AForm af;
    if (!form_of(a_form, &af)) return JSCAN_ERR_FORM;
    bool empty = false;
    jscan_status st = check_prefill(x, delta, A, B, C, h0, false, y, h_final, batch, L, D, N, dtype, &empty, af);
    if (st != JSCAN_OK) return st;
    if (chunk < -1) return JSCAN_ERR_SHAPE;
    if (chunk > 0 && af != AForm::Diagonal) return JSCAN_ERR_FORM;   // segments are composed for the diagonal form
    if (empty) return JSCAN_OK;
    const int64_t es = elem_bytes(dtype);
    if (L > 0) st = check_gate(skip, z, ld_z, y, D, h_final, batch * L, batch, D, es);
    if (st != JSCAN_OK) return st;
    GateArgs a{};
    a.x = x, a.delta = delta, a.A = A, a.B = B, a.C = C, a.h0 = h0, a.y = y, a.h_final = h_final;
    a.batch = batch, a.L = L, a.D = D, a.gate = OutGate{skip, z, ld_z}, a.stream = static_cast<hipStream_t>(stream);
    a.fp32_sum = chunk >= 0;
    if (L == 0) {
        const int64_t total = batch * D * jscan::kDState, each = (int64_t)1 << 31;
        for (int64_t i = 0; i < total; i += each) {
            const int64_t count = each < total - i ? each : total - i;
            hipLaunchKernelGGL(jscan::copy_state_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, a.stream,
                               at<float>(h0, i), h_final + i, count);
        }
        return launch_status();
    }
    ChunkPlan p;
    if (af == AForm::Diagonal && chunk >= 0) p = chunk > 0 ? plan_chunks(batch, L, D, chunk) : plan_automatic(batch, L, D);
    if (p.n_seg <= 1) {
        dispatch(dtype, af, [&](auto e, auto f) { launch_prefill<decltype(e), (AForm)decltype(f)::value>(a); });
        return launch_status();
    }
    if (!gate_grids_fit(batch, D, p)) return JSCAN_ERR_SHAPE;
    const int64_t need = chunk_workspace_bytes(p, batch, D);
    if (!workspace) return JSCAN_ERR_NULL;
    if (workspace_bytes < need) return JSCAN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return JSCAN_ERR_ALIGN;
    const int64_t seq = batch * L * D * es, bc = batch * L * N * es, state = batch * D * N * 4;
    const Rows scratch[] = {flat(workspace, need)};
    const Rows others[] = {flat(x, seq), flat(delta, seq), flat(A, D * N * 4), flat(B, bc), flat(C, bc), flat(h0, state),
                           flat(y, seq), flat(h_final, state), flat(skip, D * 4), rows_of({z, ld_z}, batch * L, D, es)};
    if (any_overlap(scratch, others)) return JSCAN_ERR_ALIAS;
    if (dtype == JSCAN_BF16) return launch_chunked<jscan::BF16>(a, p, workspace);
    return launch_chunked<jscan::F32>(a, p, workspace);
}

jscan_status jscan_step_gate(float *h, const void *x_t, const void *delta_t, const float *A, const void *B_t,
                             const void *C_t, const float *skip, const void *z_t, void *y_t, int64_t batch, int64_t D,
                             int64_t N, int64_t ld_xd, int64_t ld_bc, int64_t ld_z, int64_t ld_y, jscan_a_form a_form,
                             jscan_dtype dtype, void *stream) {
    AForm af;
    if (!form_of(a_form, &af)) return JSCAN_ERR_FORM;
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (batch < 0 || D < 0 || N != JSCAN_D_STATE || D % 8 != 0 || D > (1 << 24) || batch > (1 << 20))
        return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) return JSCAN_OK;
    if (!ld_ok(ld_xd, batch, D) || !ld_ok(ld_bc, batch, N) || !ld_ok(ld_y, batch, D) || ld_xd % 8 != 0 ||
        ld_bc % 8 != 0 || ld_y % 8 != 0)
        return JSCAN_ERR_SHAPE;
    if (!h || !x_t || !delta_t || !A || !B_t || !C_t || !y_t) return JSCAN_ERR_NULL;
    for (const void *p : {(const void *)h, x_t, delta_t, (const void *)A, B_t, C_t, (const void *)y_t})
        if (!aligned16(p)) return JSCAN_ERR_ALIGN;
    const int64_t es = elem_bytes(dtype);
    const jscan_status st = check_gate(skip, z_t, ld_z, y_t, ld_y, h, batch, batch, D, es);
    if (st != JSCAN_OK) return st;
    const Rows out[] = {flat(h, batch * D * N * 4), rows_of({y_t, ld_y}, batch, D, es)};
    const Rows in[] = {rows_of({x_t, ld_xd}, batch, D, es), rows_of({delta_t, ld_xd}, batch, D, es),
                       flat(A, D * (af == AForm::ScaledIdentity ? 1 : N) * 4), rows_of({B_t, ld_bc}, batch, N, es),
                       rows_of({C_t, ld_bc}, batch, N, es)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    GateArgs a{};
    a.h = h, a.x = x_t, a.delta = delta_t, a.A = A, a.B = B_t, a.C = C_t, a.y = y_t, a.batch = batch, a.D = D;
    a.ld_xd = ld_xd, a.ld_bc = ld_bc, a.ld_y = ld_y, a.gate = OutGate{skip, z_t, ld_z};
    a.stream = static_cast<hipStream_t>(stream);
    dispatch(dtype, af, [&](auto e, auto f) { launch_step<decltype(e), (AForm)decltype(f)::value>(a); });
    return launch_status();
}

}  // extern "C"

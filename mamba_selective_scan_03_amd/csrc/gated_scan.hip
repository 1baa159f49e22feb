// gated_scan.hip - host entry points of the gated recurrence (include/jscan.h): the scan over whole
// sequences, its backward pass and the decode step.
#include "host_common.h"
#include "gated_scan_kernels.h"

using namespace jscan::host;
using jscan::GateForm;
using jscan::TokenRows;

namespace {

bool form_ok(jscan_gate_form f) { return f == JSCAN_GATE_DECAY || f == JSCAN_GATE_SIGMOID; }

// Sizes that the index arithmetic of the kernels holds: rows of D and grids in 32 bits, byte
// offsets in 63.
bool shape_ok(int64_t batch, int64_t L, int64_t D) {
    return batch >= 0 && L >= 0 && D >= 0 && D <= (1 << 24) && batch <= (1 << 20) && L < ((int64_t)1 << 31) &&
           batch * ((D + 63) / 64) <= kMaxBlocks;
}
bool ld_ok(int64_t ld, int64_t rows, int64_t D) { return ld >= D && (rows == 0 || ld <= ((int64_t)1 << 58) / rows); }

struct Pair {
    const void *p;
    int64_t ld;
};

Rows rows_of(Pair t, int64_t rows, int64_t D, int64_t es) { return Rows{t.p, t.p ? rows : 0, D * es, t.ld * es}; }
Rows flat(const void *p, int64_t bytes) { return Rows{p, p && bytes > 0 ? 1 : 0, bytes, bytes}; }

// Whether an output shares memory with an input or with another output.
template <int NO, int NI> bool any_overlap(const Rows (&out)[NO], const Rows (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(out[i], in[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlaps(out[i], out[j])) return true;
    }
    return false;
}

template <typename E> TokenRows<const typename E::store_t> in_rows(const void *p, int64_t ld) {
    return {static_cast<const typename E::store_t *>(p), ld};
}
template <typename E> TokenRows<typename E::store_t> out_rows(void *p, int64_t ld) {
    return {static_cast<typename E::store_t *>(p), ld};
}

template <typename E, GateForm F>
jscan_status launch_scan(const void *g, const void *u, const float *h0, const int32_t *lengths, void *y,
                         float *h_final, int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u,
                         int64_t ld_y, hipStream_t s) {
    const int strips = (int)((D + 63) / 64);
    hipLaunchKernelGGL((jscan::gated_lane_kernel<E, F>), dim3((unsigned)(batch * strips)), dim3(64), 0, s,
                       in_rows<E>(g, ld_g), in_rows<E>(u, ld_u), h0, lengths, out_rows<E>(y, ld_y), h_final, L,
                       (int)D, strips);
    return launch_status();
}

template <typename E, GateForm F>
jscan_status launch_backward(const void *g, const void *u, const void *y, const void *dy, const float *h0,
                             const float *dh_final, const int32_t *lengths, void *dg, void *du, float *dh0,
                             int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u, int64_t ld_y,
                             int64_t ld_dy, int64_t ld_dg, int64_t ld_du, hipStream_t s) {
    const int strips = (int)((D + 63) / 64);
    hipLaunchKernelGGL((jscan::gated_lane_backward_kernel<E, F>), dim3((unsigned)(batch * strips)), dim3(64), 0, s,
                       in_rows<E>(g, ld_g), in_rows<E>(u, ld_u), in_rows<E>(y, ld_y), in_rows<E>(dy, ld_dy), h0,
                       dh_final, lengths, out_rows<E>(dg, ld_dg), out_rows<E>(du, ld_du), dh0, L, (int)D, strips);
    return launch_status();
}

template <typename E, GateForm F>
jscan_status launch_step(float *h, const void *g, const void *u, void *y, int64_t batch, int64_t D, int64_t ld_g,
                         int64_t ld_u, int64_t ld_y, hipStream_t s) {
    using T = typename E::store_t;
    const int blocks = (int)((D + 255) / 256);
    hipLaunchKernelGGL((jscan::gated_step_kernel<E, F>), dim3((unsigned)(batch * blocks)), dim3(256), 0, s, h,
                       static_cast<const T *>(g), static_cast<const T *>(u), static_cast<T *>(y), (int)D, blocks,
                       ld_g, ld_u, ld_y);
    return launch_status();
}

// Calls f with the element and form types that dtype and form name.
template <typename Fn> jscan_status dispatch(jscan_dtype dtype, jscan_gate_form form, Fn f) {
    using Decay = std::integral_constant<GateForm, GateForm::Decay>;
    using Sigmoid = std::integral_constant<GateForm, GateForm::Sigmoid>;
    if (dtype == JSCAN_BF16) return form == JSCAN_GATE_DECAY ? f(jscan::BF16{}, Decay{}) : f(jscan::BF16{}, Sigmoid{});
    return form == JSCAN_GATE_DECAY ? f(jscan::F32{}, Decay{}) : f(jscan::F32{}, Sigmoid{});
}

}  // namespace

extern "C" {

int64_t jscan_gated_scan_workspace(int64_t batch, int64_t L, int64_t D) {
    if (!shape_ok(batch, L, D)) return -1;
    return 0;
}

jscan_status jscan_gated_scan(const void *g, const void *u, const float *h0, const int32_t *lengths, void *y,
                              float *h_final, int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u,
                              int64_t ld_y, void *workspace, int64_t workspace_bytes, jscan_gate_form form,
                              jscan_dtype dtype, void *stream) {
    if (!form_ok(form)) return JSCAN_ERR_FORM;
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!shape_ok(batch, L, D)) return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) return JSCAN_OK;
    const int64_t tokens = batch * L, es = elem_bytes(dtype), state = batch * D * 4;
    if (L > 0 && !(ld_ok(ld_g, tokens, D) && ld_ok(ld_u, tokens, D) && ld_ok(ld_y, tokens, D))) return JSCAN_ERR_SHAPE;
    if (!h_final || (L > 0 && (!g || !u || !y))) return JSCAN_ERR_NULL;
    const int64_t need = jscan_gated_scan_workspace(batch, L, D);
    if (need > 0 && !workspace) return JSCAN_ERR_NULL;
    if (need > 0 && workspace_bytes < need) return JSCAN_ERR_WORKSPACE;
    if (!aligned(g, es) || !aligned(u, es) || !aligned(y, es) || !aligned(h0, 4) || !aligned(h_final, 4) ||
        !aligned(lengths, 4) || (need > 0 && !aligned16(workspace)))
        return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of({y, ld_y}, tokens, D, es), flat(h_final, state), flat(workspace, need)};
    const Rows in[] = {rows_of({g, ld_g}, tokens, D, es), rows_of({u, ld_u}, tokens, D, es),
                       flat(h0 == h_final ? nullptr : h0, state), flat(lengths, batch * 4)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dispatch(dtype, form, [&](auto e, auto f) {
        return launch_scan<decltype(e), decltype(f)::value>(g, u, h0, lengths, y, h_final, batch, L, D, ld_g, ld_u,
                                                            ld_y, s);
    });
}

jscan_status jscan_gated_scan_backward(const void *g, const void *u, const void *y, const void *dy, const float *h0,
                                       const float *dh_final, const int32_t *lengths, void *dg, void *du, float *dh0,
                                       int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u, int64_t ld_y,
                                       int64_t ld_dy, int64_t ld_dg, int64_t ld_du, void *workspace,
                                       int64_t workspace_bytes, jscan_gate_form form, jscan_dtype dtype,
                                       void *stream) {
    if (!form_ok(form)) return JSCAN_ERR_FORM;
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!shape_ok(batch, L, D)) return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) return JSCAN_OK;
    const int64_t tokens = batch * L, es = elem_bytes(dtype), state = batch * D * 4;
    const bool sig = form == JSCAN_GATE_SIGMOID;   // the decay form does not read u
    if (L > 0) {
        const int64_t lds[] = {ld_g, ld_y, ld_dy, ld_dg, ld_du, sig ? ld_u : D};
        for (int64_t ld : lds)
            if (!ld_ok(ld, tokens, D)) return JSCAN_ERR_SHAPE;
        if (!g || !y || !dy || !dg || !du || (sig && !u)) return JSCAN_ERR_NULL;
    }
    const int64_t need = jscan_gated_scan_workspace(batch, L, D);
    if (need > 0 && !workspace) return JSCAN_ERR_NULL;
    if (need > 0 && workspace_bytes < need) return JSCAN_ERR_WORKSPACE;
    const void *elems[] = {g, sig ? u : nullptr, y, dy, dg, du};
    for (const void *p : elems)
        if (!aligned(p, es)) return JSCAN_ERR_ALIGN;
    if (!aligned(h0, 4) || !aligned(dh_final, 4) || !aligned(dh0, 4) || !aligned(lengths, 4) ||
        (need > 0 && !aligned16(workspace)))
        return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of({dg, ld_dg}, tokens, D, es), rows_of({du, ld_du}, tokens, D, es), flat(dh0, state),
                        flat(workspace, need)};
    const Rows in[] = {rows_of({g, ld_g}, tokens, D, es),   rows_of({sig ? u : nullptr, ld_u}, tokens, D, es),
                       rows_of({y, ld_y}, tokens, D, es),   rows_of({dy, ld_dy}, tokens, D, es),
                       flat(h0, state),                     flat(dh_final == dh0 ? nullptr : dh_final, state),
                       flat(lengths, batch * 4)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dispatch(dtype, form, [&](auto e, auto f) {
        return launch_backward<decltype(e), decltype(f)::value>(g, u, y, dy, h0, dh_final, lengths, dg, du, dh0, batch,
                                                                L, D, ld_g, ld_u, ld_y, ld_dy, ld_dg, ld_du, s);
    });
}

jscan_status jscan_gated_step(float *h, const void *g_t, const void *u_t, void *y_t, int64_t batch, int64_t D,
                              int64_t ld_g, int64_t ld_u, int64_t ld_y, jscan_gate_form form, jscan_dtype dtype,
                              void *stream) {
    if (!form_ok(form)) return JSCAN_ERR_FORM;
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (!shape_ok(batch, 1, D)) return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) return JSCAN_OK;
    if (!(ld_ok(ld_g, batch, D) && ld_ok(ld_u, batch, D) && ld_ok(ld_y, batch, D))) return JSCAN_ERR_SHAPE;
    if (!h || !g_t || !u_t || !y_t) return JSCAN_ERR_NULL;
    const int64_t es = elem_bytes(dtype);
    if (!aligned(g_t, es) || !aligned(u_t, es) || !aligned(y_t, es) || !aligned(h, 4)) return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of({y_t, ld_y}, batch, D, es), flat(h, batch * D * 4)};
    const Rows in[] = {rows_of({g_t, ld_g}, batch, D, es), rows_of({u_t, ld_u}, batch, D, es)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dispatch(dtype, form, [&](auto e, auto f) {
        return launch_step<decltype(e), decltype(f)::value>(h, g_t, u_t, y_t, batch, D, ld_g, ld_u, ld_y, s);
    });
}

}  // extern "C"

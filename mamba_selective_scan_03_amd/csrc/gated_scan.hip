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

// How a call is laid out: strips of `lanes` lanes, `waves` waves a work-group, n_seg segments of seg_len tokens.
struct Plan {
    int lanes, waves;
    int64_t n_seg, seg_len;
    bool stream = false;   // with the non-temporal hint
};

constexpr int kRun = 8;   // tokens a thread takes of a block, and between two saved states

int64_t state_rows(int64_t L) { return (L + kRun - 1) / kRun; }

// Narrower strips and segments both make more work-groups.  Narrow strips read every byte once but in
// pieces of 64 or 128 bytes a row, and a work-group has less in flight; segments read two of the tensors
// twice (the maps first), with a second launch.  The layout is the one with the least expected time,
//     sqrt(memory^2 + chain^2), and 7 us more when cut,
// where memory is the bytes at the rates that large scans reach (5.3 TB/s; 6.5 TB/s for what is read twice)
// and chain is the time along the tokens of one CU's work-groups, taken from single ones (1 x 65536 x 1024:
// 6.0, 3.8, 3.0 ns a token and tensor for 64, 32, 16 lanes).  What it chooses between, measured (us):
//     2 x 4096 x 4096 sigmoid   forward   64 lanes 102, 32 lanes 65, 16 lanes 54, 64 lanes in 4 segments 57
//                               backward  64 lanes 180, 32 lanes 119, 16 lanes 108, 64 lanes in 4 segments 95
//     24 x 1000 x 500           forward   64 lanes 26.5, 32 lanes 19.6, 16 lanes 23.6
//     1 x 65536 x 1024          forward   16 lanes 609, 64 lanes in 32 segments 118, in 64 segments 121
//     39 x 13148 x 184 sigmoid  backward  16 lanes 287, 64 lanes in 2 segments 537, in 3 segments 423
// Over 630 scans and backward passes of random sizes its choice is 1.4% slower than the best layout tried, which itself
// may be well off the passes' bytes (profiles/sweep_gated_scan_layouts.txt has every time).
// Where strips of 64 lanes are more than the chip holds at a time (512, two work-groups a CU), what counts is how
// little of a block lies behind a short sequence's end (one wave takes 8 tokens a block, four 32, eight 64,
// narrow strips of 32 lanes 128), and for long ones how evenly the turns end (us for 64 and 32 lanes: 75 x 1500
// x 1000 sigmoid 170 and 159, backward 330 and 314; 38 x 1500 x 2048 decay 146 and 128, 247 and 225; 16 x 4096 x
// 8192 621 and 580; at 512 strips, 32 x 1500 x 2048 sigmoid 117 and 119, 229 and 235; at 600 tokens, 75 x 600 x 1000
// 55 and 62). From 257 tokens on, over 280 passes of 300 to 4096 tokens and 300 to 3000 strips this choice is 1.6%
// slower than the better of the two:
//     36 x 36 x 8832            forward   one wave 13, four 16, eight 20, 32 lanes 45;       backward  21, 26, 48, 75
//     497 x 123 x 2016 sigmoid  forward   one wave 157, four 141, eight 143, 32 lanes 235;   backward  310, 284, 318, 395
//     108 x 157 x 7161          forward   one wave 167, four 154, eight 168, 32 lanes 230;   backward  289, 274, 336, 494
//     72 x 379 x 3810 fp32 sig. forward   one wave 284, four 264, eight 251, 32 lanes 257;   backward  659, 560, 506, 546
// and sequences of a few tokens take few waves everywhere (256 x 8 x 4096: one wave 10.8 us, four 23 us).
// channels: per lane.  tensors: rows of D elements moved per token.  narrow: whether the lane offsets of
// narrow strips fit 32 bits.
constexpr int64_t kLeastSegment = 256;   // tokens
constexpr int64_t kMostGroups = 768;     // work-groups that cutting makes, at most
constexpr int64_t kWideAtOnce = 512;     // work-groups of 64 lanes that run at a time

Plan plan_for(int64_t batch, int64_t L, int64_t D, int channels, int es, int tensors, bool narrow) {
    auto groups_of = [&](int lanes) { return batch * ((D + lanes * channels - 1) / (lanes * channels)); };
    const int64_t wide = groups_of(64);
    if (L <= kRun || (L <= 8 * kRun && wide >= 768)) return {64, 1, 1, L};
    if (L <= 4 * kRun || (L <= 32 * kRun && wide >= 256)) return {64, 4, 1, L};
    if (narrow && wide > kWideAtOnce) return {L < 1024 ? 64 : 32, 8, 1, L};
    constexpr int kLanes[] = {64, 32, 16};
    constexpr float kToken[] = {6.0e-3f, 3.8e-3f, 3.0e-3f};
    const float elements = (float)(batch * L) * (float)D, once = elements * (float)(es * tensors) / 5.3e6f;
    const float twice = elements * (float)(2 * es) / 6.5e6f;
    Plan best{64, 8, 1, L};
    float least = 0.0f;
    for (int i = 0; i < (narrow ? 3 : 1); ++i) {
        const int lanes = kLanes[i];
        if (lanes > 16 && narrow && D <= lanes * channels / 2) continue;   // half the lanes would repeat a channel
        const int64_t groups = groups_of(lanes);
        const float token = kToken[i] * (float)tensors;
        const int64_t block = (int64_t)(64 / lanes) * 8 * kRun;
        auto consider = [&](int64_t n) {
            const int64_t seg = n == 1 ? L : ((L + n - 1) / n + block - 1) / block * block, n_seg = (L + seg - 1) / seg;
            const float chain = (float)((groups * n_seg + 255) / 256) * (float)seg * token;
            const float memory = n_seg == 1 ? once : once + twice;
            const float us = __builtin_sqrtf(memory * memory + chain * chain) + (n_seg == 1 ? 0.0f : 7.0f);
            if (least == 0.0f || us < least) {
                least = us;
                best = {lanes, 8, n_seg, seg};
            }
        };
        consider(1);
        if (lanes == 32) continue;
        for (int64_t want = 128; want <= kMostGroups; want += 128)
            for (int64_t up = 0; up < 2; ++up) {   // just below and just above whole and half rounds of the CUs
                int64_t n = want / groups + up;
                n = n < L / kLeastSegment ? n : L / kLeastSegment;
                if (n > 1 && n * groups <= kMostGroups) consider(n);
            }
    }
    return best;
}

// Enough for any plan: strips of 64 lanes with two channels make the fewest work-groups and so the most segments.
int64_t most_segments(int64_t batch, int64_t L, int64_t D) {
    const int64_t n = kMostGroups / (batch * ((D + 127) / 128));
    return n < L / kLeastSegment ? n : L / kLeastSegment;
}

int64_t workspace_bytes_for(int64_t batch, int64_t L, int64_t D) {
    const int64_t n = most_segments(batch, L, D);
    return n > 1 ? batch * D * (n * 8 + 4) : 0;
}

jscan::SegSplit split_of(const Plan &p, int64_t batch, int64_t D, void *workspace) {
    float2 *sums = static_cast<float2 *>(workspace);
    return {(int)p.n_seg, p.seg_len, sums, reinterpret_cast<float *>(sums + batch * D * p.n_seg)};
}

template <typename V> TokenRows<const typename V::store_t> in_rows(Pair t) {
    return {static_cast<const typename V::store_t *>(t.p), t.ld};
}
template <typename V> TokenRows<typename V::store_t> out_rows(Pair t) {
    return {static_cast<typename V::store_t *>(const_cast<void *>(t.p)), t.ld};
}

Pair from_row(Pair t, int64_t row, int64_t es) {
    return {t.p ? static_cast<const char *>(t.p) + row * t.ld * es : nullptr, t.ld};
}
template <typename T> T *from(T *p, int64_t i) { return p ? p + i : nullptr; }

struct ScanArgs {
    Pair g, u, y;
    const float *h0;
    const int32_t *lengths;
    float *h_final, *states;   // states: NULL unless saved
    int64_t batch, L, D;
    void *workspace;
    hipStream_t stream;

    ScanArgs sequences(int64_t b, int64_t n, int64_t es) const {   // the call on sequences b .. b + n - 1
        return {from_row(g, b * L, es), from_row(u, b * L, es), from_row(y, b * L, es), from(h0, b * D),
                from(lengths, b),       from(h_final, b * D),   from(states, b * state_rows(L) * D),
                n, L, D, workspace, stream};
    }
};

struct BackwardArgs {
    Pair g, u, y, dy, dg, du;
    const float *h0, *states, *dh_final;   // states in place of y and h0 when saved
    const int32_t *lengths;
    float *dh0;
    int64_t batch, L, D;
    void *workspace;
    hipStream_t stream;

    BackwardArgs sequences(int64_t b, int64_t n, int64_t es) const {
        return {from_row(g, b * L, es),  from_row(u, b * L, es),  from_row(y, b * L, es), from_row(dy, b * L, es),
                from_row(dg, b * L, es), from_row(du, b * L, es), from(h0, b * D),
                from(states, b * state_rows(L) * D), from(dh_final, b * D), from(lengths, b), from(dh0, b * D),
                n, L, D, workspace, stream};
    }
};

template <typename V, GateForm F, int LC, int NW, bool kRev, bool kSaved>
void launch_summary(Pair g, Pair x, const float *s0, const int32_t *lengths, const jscan::SegSplit &sp, int64_t batch,
                    int64_t L, int64_t D, hipStream_t stream) {
    const int strips = (int)((D + LC * V::n - 1) / (LC * V::n));
    hipLaunchKernelGGL((jscan::gated_summary_kernel<V, F, LC, NW, kRun, kRev, kRev && kSaved>),
                       dim3((unsigned)(batch * strips * (sp.n_seg - 1))), dim3(NW * 64), 0, stream, in_rows<V>(g),
                       in_rows<V>(x), s0, lengths, sp, L, (int)D, strips);
}

template <typename V, GateForm F, int LC, int NW, bool kNt, bool kSaved> void launch_as(const ScanArgs &a, const Plan &p) {
    const int strips = (int)((a.D + LC * V::n - 1) / (LC * V::n));
    const jscan::SegSplit sp = split_of(p, a.batch, a.D, a.workspace);
    if constexpr (NW == 8 && LC != 32) {
        if (p.n_seg > 1)
            launch_summary<V, F, LC, NW, false, kSaved>(a.g, a.u, a.h0, a.lengths, sp, a.batch, a.L, a.D, a.stream);
    }
    hipLaunchKernelGGL((jscan::gated_scan_kernel<V, F, LC, NW, kRun, kNt, kSaved>),
                       dim3((unsigned)(a.batch * strips * p.n_seg)), dim3(NW * 64), 0, a.stream, in_rows<V>(a.g),
                       in_rows<V>(a.u), a.h0, a.lengths, out_rows<V>(a.y), a.h_final, a.states, sp, a.L, (int)a.D, strips);
}

template <typename V, GateForm F, int LC, int NW, bool kNt, bool kSaved> void launch_as(const BackwardArgs &a, const Plan &p) {
    const int strips = (int)((a.D + LC * V::n - 1) / (LC * V::n));
    const jscan::SegSplit sp = split_of(p, a.batch, a.D, a.workspace);
    if constexpr (NW == 8 && LC != 32) {
        if (p.n_seg > 1)
            launch_summary<V, F, LC, NW, true, kSaved>(a.g, a.dy, a.dh_final, a.lengths, sp, a.batch, a.L, a.D, a.stream);
    }
    hipLaunchKernelGGL((jscan::gated_backward_kernel<V, F, LC, NW, kRun, kNt, kSaved>),
                       dim3((unsigned)(a.batch * strips * p.n_seg)), dim3(NW * 64), 0, a.stream, in_rows<V>(a.g),
                       in_rows<V>(a.u), in_rows<V>(a.y), in_rows<V>(a.dy), a.h0, a.states, a.dh_final, a.lengths,
                       out_rows<V>(a.dg), out_rows<V>(a.du), a.dh0, sp, a.L, (int)a.D, strips);
}

template <typename V, GateForm F, bool kS, typename Args> void launch_plan(const Args &a, const Plan &p) {
    if (p.waves == 1) launch_as<V, F, 64, 1, false, kS>(a, p);
    else if (p.waves == 4) launch_as<V, F, 64, 4, false, kS>(a, p);
    else if (p.lanes == 64) p.stream ? launch_as<V, F, 64, 8, true, kS>(a, p) : launch_as<V, F, 64, 8, false, kS>(a, p);
    else if (p.lanes == 32) p.stream ? launch_as<V, F, 32, 8, true, kS>(a, p) : launch_as<V, F, 32, 8, false, kS>(a, p);
    else launch_as<V, F, 16, 8, false, kS>(a, p);
}

// Whether every row of a call's tensors starts on 4 bytes and holds an even number of bf16 values.
template <int N> bool two_channels(const Pair (&t)[N], int64_t D) {
    if (D % 2) return false;
    for (const Pair &r : t)
        if (r.p && (r.ld % 2 || !aligned(r.p, 4))) return false;
    return true;
}
// Whether the lane offsets of narrow strips (three runs of kRun rows, and the row itself) fit 32 bits.
template <int N> bool narrow_ok(const Pair (&t)[N], int64_t es) {
    for (const Pair &r : t)
        if (r.p && r.ld * es > ((int64_t)1 << 31) / (4 * kRun)) return false;
    return true;
}

// Whether every row of a call's tensors starts on a line of 128 bytes.
template <int N> bool whole_lines(const Pair (&t)[N], int64_t es) {
    for (const Pair &r : t)
        if (r.p && (r.ld * es % 128 || !aligned(r.p, 128))) return false;
    return true;
}

// More than the last-level cache holds (256 MB) goes by with the non-temporal hint where rows are whole
// lines (16 x 4096 x 8192: 583 us against 620 us without, backward 1198 and 1265 us; 1 x 65536 x 1024: 120
// and 132, 160 and 192 us). Rows that share lines want them kept for the neighbouring strip (3 x 6225 x
// 3864: 123 us with, 115 us without, backward 283 and 248 us), and less data may be in the cache already (2
// x 4096 x 4096 repeated: 55 us with, 38 us without).
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// kSaved: with saved states (bf16 only).
template <bool kSaved, typename Args, int N>
jscan_status launch_args(const Args &a, const Pair (&t)[N], jscan_dtype dtype, jscan_gate_form form, bool backward) {
    const bool two = dtype == JSCAN_BF16 && two_channels(t, a.D);
    const int tensors = !backward ? 3 : form == JSCAN_GATE_SIGMOID && !kSaved ? 6 : 5;
    const int64_t es = elem_bytes(dtype);
    Plan p = plan_for(a.batch, a.L, a.D, two ? 2 : 1, (int)es, tensors, narrow_ok(t, es));
    p.stream = whole_lines(t, es) && a.batch * a.L * a.D * es * tensors > kStreamBytes;
    // a plan's work-items per sequence; as many sequences a launch as it can count (all but for
    // enormous batches, whose tokens are not cut)
    const int64_t channels = two ? 2 : 1, strips = (a.D + p.lanes * channels - 1) / (p.lanes * channels);
    const int64_t most = kMaxItems / (strips * p.n_seg * p.waves * 64);
    auto with_form = [&](auto v) {
        using V = decltype(v);
        for (int64_t b = 0; b < a.batch; b += most) {
            const Args part = b == 0 && a.batch <= most ? a : a.sequences(b, a.batch - b < most ? a.batch - b : most, es);
            if (form == JSCAN_GATE_DECAY) launch_plan<V, GateForm::Decay, kSaved>(part, p);
            else launch_plan<V, GateForm::Sigmoid, kSaved>(part, p);
        }
    };
    if (two) with_form(jscan::Bf16x2{});
    else if (kSaved || dtype == JSCAN_BF16) with_form(jscan::Bf16x1{});
    else if constexpr (!kSaved) with_form(jscan::F32x1{});
    return launch_status();
}

// The checks of a scan and its launch.  states: where they are saved, of which a call without tokens has none.
template <bool kSaved>
jscan_status scan(const ScanArgs &a, int64_t workspace_bytes, jscan_gate_form form, jscan_dtype dtype) {
    if (!form_ok(form)) return JSCAN_ERR_FORM;
    if (dtype != JSCAN_BF16 && (kSaved || dtype != JSCAN_F32)) return JSCAN_ERR_DTYPE;
    if (!shape_ok(a.batch, a.L, a.D)) return JSCAN_ERR_SHAPE;
    if (a.batch == 0 || a.D == 0) return JSCAN_OK;
    const int64_t tokens = a.batch * a.L, es = elem_bytes(dtype), state = a.batch * a.D * 4;
    const Pair t[] = {a.g, a.u, a.y};
    if (a.L > 0) {
        for (const Pair &p : t)
            if (!ld_ok(p.ld, tokens, a.D)) return JSCAN_ERR_SHAPE;
        if (!a.g.p || !a.u.p || !a.y.p || (kSaved && !a.states)) return JSCAN_ERR_NULL;
    }
    if (!a.h_final) return JSCAN_ERR_NULL;
    const int64_t need = workspace_bytes_for(a.batch, a.L, a.D);
    if (need > 0 && !a.workspace) return JSCAN_ERR_NULL;
    if (need > 0 && workspace_bytes < need) return JSCAN_ERR_WORKSPACE;
    for (const Pair &p : t)
        if (!aligned(p.p, es)) return JSCAN_ERR_ALIGN;
    if (!aligned(a.h0, 4) || !aligned(a.h_final, 4) || !aligned(a.lengths, 4) || !aligned16(a.states) ||
        (need > 0 && !aligned16(a.workspace)))
        return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of(a.y, tokens, a.D, es), flat(a.h_final, state), flat(a.workspace, need),
                        flat(a.states, state * state_rows(a.L))};
    const Rows in[] = {rows_of(a.g, tokens, a.D, es), rows_of(a.u, tokens, a.D, es),
                       flat(a.h0 == a.h_final ? nullptr : a.h0, state), flat(a.lengths, a.batch * 4)};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    return launch_args<kSaved>(a, t, dtype, form, false);
}

// The same for a backward pass.
template <bool kSaved>
jscan_status backward(BackwardArgs a, int64_t workspace_bytes, jscan_gate_form form, jscan_dtype dtype) {
    if (!form_ok(form)) return JSCAN_ERR_FORM;
    if (dtype != JSCAN_BF16 && (kSaved || dtype != JSCAN_F32)) return JSCAN_ERR_DTYPE;
    if (!shape_ok(a.batch, a.L, a.D)) return JSCAN_ERR_SHAPE;
    if (a.batch == 0 || a.D == 0) return JSCAN_OK;
    const int64_t tokens = a.batch * a.L, es = elem_bytes(dtype), state = a.batch * a.D * 4;
    const bool reads_u = kSaved || form == JSCAN_GATE_SIGMOID;   // from y, the decay form does not
    if (!reads_u) a.u = {nullptr, a.D};
    const Pair t[] = {a.g, a.u, a.y, a.dy, a.dg, a.du};
    if (a.L > 0) {
        for (const Pair &p : t)
            if (!ld_ok(p.ld, tokens, a.D)) return JSCAN_ERR_SHAPE;
        if (!a.g.p || !(kSaved ? (const void *)a.states : a.y.p) || !a.dy.p || !a.dg.p || !a.du.p || (reads_u && !a.u.p))
            return JSCAN_ERR_NULL;
    }
    const int64_t need = workspace_bytes_for(a.batch, a.L, a.D);
    if (need > 0 && !a.workspace) return JSCAN_ERR_NULL;
    if (need > 0 && workspace_bytes < need) return JSCAN_ERR_WORKSPACE;
    for (const Pair &p : t)
        if (!aligned(p.p, es)) return JSCAN_ERR_ALIGN;
    if (!aligned(a.h0, 4) || !aligned(a.dh_final, 4) || !aligned(a.dh0, 4) || !aligned(a.lengths, 4) ||
        !aligned16(a.states) || (need > 0 && !aligned16(a.workspace)))
        return JSCAN_ERR_ALIGN;
    const Rows out[] = {rows_of(a.dg, tokens, a.D, es), rows_of(a.du, tokens, a.D, es), flat(a.dh0, state),
                        flat(a.workspace, need)};
    const Rows in[] = {rows_of(a.g, tokens, a.D, es),  rows_of(a.u, tokens, a.D, es),
                       rows_of(a.y, tokens, a.D, es),  rows_of(a.dy, tokens, a.D, es),
                       flat(a.h0, state),              flat(a.dh_final == a.dh0 ? nullptr : a.dh_final, state),
                       flat(a.lengths, a.batch * 4),   flat(a.states, state * state_rows(a.L))};
    if (any_overlap(out, in)) return JSCAN_ERR_ALIAS;
    return launch_args<kSaved>(a, t, dtype, form, true);
}

// Four channels a thread where D, the strides and the addresses allow it (256 x 8192 bf16 5.1 us, 5.8 TB/s), or one
// (256 x 8191: 6.9 us).
template <typename E, GateForm F>
jscan_status launch_step(float *h, const void *g, const void *u, void *y, int64_t batch, int64_t D, int64_t ld_g,
                         int64_t ld_u, int64_t ld_y, hipStream_t s) {
    using T = typename E::store_t;
    constexpr int64_t kVec = 4, kBytes = kVec * (int64_t)sizeof(T);
    const T *gt = static_cast<const T *>(g), *ut = static_cast<const T *>(u);
    T *yt = static_cast<T *>(y);
    const bool wide = D % kVec == 0 && ld_g % kVec == 0 && ld_u % kVec == 0 && ld_y % kVec == 0 && aligned(g, kBytes) &&
                      aligned(u, kBytes) && aligned(y, kBytes) && aligned16(h);
    const int64_t per = wide ? 256 * kVec : 256, blocks = (D + per - 1) / per, most = kMaxItems / (blocks * 256);
    for (int64_t b = 0; b < batch; b += most) {   // as many sequences a launch as it can count
        const dim3 grid((unsigned)((batch - b < most ? batch - b : most) * blocks));
        const T *gb = gt + b * ld_g, *ub = ut + b * ld_u;
        if (wide)
            hipLaunchKernelGGL((jscan::gated_step_kernel<E, F, (int)kVec>), grid, dim3(256), 0, s, h + b * D, gb, ub,
                               yt + b * ld_y, (int)D, (int)blocks, ld_g, ld_u, ld_y);
        else
            hipLaunchKernelGGL((jscan::gated_step_kernel<E, F, 1>), grid, dim3(256), 0, s, h + b * D, gb, ub,
                               yt + b * ld_y, (int)D, (int)blocks, ld_g, ld_u, ld_y);
    }
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
    if (batch == 0 || D == 0) return 0;
    return workspace_bytes_for(batch, L, D);
}

jscan_status jscan_gated_scan(const void *g, const void *u, const float *h0, const int32_t *lengths, void *y,
                              float *h_final, int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u,
                              int64_t ld_y, void *workspace, int64_t workspace_bytes, jscan_gate_form form,
                              jscan_dtype dtype, void *stream) {
    return scan<false>({{g, ld_g}, {u, ld_u}, {y, ld_y}, h0, lengths, h_final, nullptr, batch, L, D, workspace,
                        static_cast<hipStream_t>(stream)}, workspace_bytes, form, dtype);
}

int64_t jscan_gated_scan_states(int64_t batch, int64_t L, int64_t D) {
    if (!shape_ok(batch, L, D)) return -1;
    const int64_t rows = batch * state_rows(L);
    return D > 0 && rows > ((int64_t)1 << 58) / D ? -1 : rows * D * 4;
}

jscan_status jscan_gated_scan_save(const void *g, const void *u, const float *h0, const int32_t *lengths, void *y,
                                   float *h_final, float *states, int64_t batch, int64_t L, int64_t D, int64_t ld_g,
                                   int64_t ld_u, int64_t ld_y, void *workspace, int64_t workspace_bytes,
                                   jscan_gate_form form, jscan_dtype dtype, void *stream) {
    return scan<true>({{g, ld_g}, {u, ld_u}, {y, ld_y}, h0, lengths, h_final, states, batch, L, D, workspace,
                       static_cast<hipStream_t>(stream)}, workspace_bytes, form, dtype);
}

jscan_status jscan_gated_scan_backward(const void *g, const void *u, const void *y, const void *dy, const float *h0,
                                       const float *dh_final, const int32_t *lengths, void *dg, void *du, float *dh0,
                                       int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u, int64_t ld_y,
                                       int64_t ld_dy, int64_t ld_dg, int64_t ld_du, void *workspace,
                                       int64_t workspace_bytes, jscan_gate_form form, jscan_dtype dtype,
                                       void *stream) {
    return backward<false>({{g, ld_g}, {u, ld_u}, {y, ld_y}, {dy, ld_dy}, {dg, ld_dg}, {du, ld_du}, h0, nullptr, dh_final,
                            lengths, dh0, batch, L, D, workspace, static_cast<hipStream_t>(stream)},
                           workspace_bytes, form, dtype);
}

jscan_status jscan_gated_scan_backward_saved(const void *g, const void *u, const float *states, const void *dy,
                                             const float *dh_final, const int32_t *lengths, void *dg, void *du,
                                             float *dh0, int64_t batch, int64_t L, int64_t D, int64_t ld_g,
                                             int64_t ld_u, int64_t ld_dy, int64_t ld_dg, int64_t ld_du,
                                             void *workspace, int64_t workspace_bytes, jscan_gate_form form,
                                             jscan_dtype dtype, void *stream) {
    return backward<true>({{g, ld_g}, {u, ld_u}, {nullptr, D}, {dy, ld_dy}, {dg, ld_dg}, {du, ld_du}, nullptr, states,
                           dh_final, lengths, dh0, batch, L, D, workspace, static_cast<hipStream_t>(stream)},
                          workspace_bytes, form, dtype);
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

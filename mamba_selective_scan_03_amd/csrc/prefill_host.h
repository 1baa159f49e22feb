// prefill_host.h - what the host entry points of the selective scan's prefill share: the checks of their arguments, the
// form of A, and how a time-parallel prefill is cut.
#pragma once

#include "host_common.h"
#include "prefill_rows_kernel.h"
#include "chunk_carry_kernel.h"
#include "prefill_seg_lane_kernel.h"

namespace jscan {
namespace host {

inline bool form_of(jscan_a_form f, jscan::AForm *af) {
    switch (f) {
    case JSCAN_A_DIAGONAL: *af = jscan::AForm::Diagonal; return true;
    case JSCAN_A_SCALED_IDENTITY: *af = jscan::AForm::ScaledIdentity; return true;
    case JSCAN_A_COMPLEX: *af = jscan::AForm::ComplexPairs; return true;
    }
    return false;
}

// Argument checks shared by every prefill entry point.  af: the form of A, which fixes its
// size (D values for the scaled identity, D * N otherwise).  Sets *nothing_to_do for zero-sized
// work (which is then OK without a launch).
inline jscan_status check_prefill(const void *x, const void *delta, const float *A, const void *B, const void *C,
                                  const float *h0, bool h0_required, const void *y, const float *h_final, int64_t batch,
                                  int64_t L, int64_t D, int64_t N, jscan_dtype dtype, bool *nothing_to_do,
                                  jscan::AForm af = jscan::AForm::Diagonal) {
    *nothing_to_do = false;
    if (dtype != JSCAN_F32 && dtype != JSCAN_BF16) return JSCAN_ERR_DTYPE;
    if (batch < 0 || L < 0 || D < 0 || N != JSCAN_D_STATE || D % 8 != 0) return JSCAN_ERR_SHAPE;
    // index arithmetic inside the kernels: rows of D fit in int, grid sizes in 32 bits
    if (D > (1 << 24) || batch > (1 << 20) || batch * ((D + 63) / 64) > kMaxBlocks) return JSCAN_ERR_SHAPE;
    // the state-wide kernels (empty-sequence copy, segment carry) run one thread per element
    if (batch * D * JSCAN_D_STATE / 256 > kMaxBlocks) return JSCAN_ERR_SHAPE;
    if (batch == 0 || D == 0) {
        *nothing_to_do = true;
        return JSCAN_OK;
    }
    if (!A || !h_final || (h0_required && !h0)) return JSCAN_ERR_NULL;
    if (L > 0 && (!x || !delta || !B || !C || !y)) return JSCAN_ERR_NULL;

    const int64_t es = elem_bytes(dtype);
    const void *arrays[] = {x, delta, A, B, C, h0, y, h_final};
    for (const void *p : arrays)
        if (p && !aligned16(p)) return JSCAN_ERR_ALIGN;

    const int64_t seq = batch * L * D * es, bc = batch * L * N * es;
    const int64_t state = batch * D * N * 4, a_bytes = D * (af == jscan::AForm::ScaledIdentity ? 1 : N) * 4;
    const Span sy = span(y, L > 0 ? seq : 0), sh = span(h_final, state);
    const Span inputs[] = {span(x, seq), span(delta, seq), span(A, a_bytes), span(B, bc), span(C, bc)};
    for (const Span &s : inputs)
        if (overlaps(sy, s) || overlaps(sh, s)) return JSCAN_ERR_ALIAS;
    if (overlaps(sy, sh)) return JSCAN_ERR_ALIAS;
    if (h0) {
        const Span s0 = span(h0, state);
        if (overlaps(sy, s0)) return JSCAN_ERR_ALIAS;
        if (overlaps(sh, s0) && h0 != h_final) return JSCAN_ERR_ALIAS;  // exact in-place is allowed
    }
    return JSCAN_OK;
}

struct ChunkPlan {
    int64_t seg_len = 0;
    int64_t n_seg = 1;
};

// Segments of `chunk` tokens, or (chunk == 0) as many as it takes to give the segment-lane
// kernel kSegLanes (segment, channel) lanes, four waves on each of the 1024 SIMDs, when the
// sequences' channels are too few for the token-by-token kernel to fill the GPU (fewer than
// 8192 channels, or D not a multiple of 32).  Automatic segments are at least 256 tokens long
// and a multiple of 64.
constexpr int64_t kSegLanes = (int64_t)1024 * jscan::seglane::kWavesPerSimd * 64;
inline ChunkPlan plan_chunks(int64_t batch, int64_t L, int64_t D, int64_t chunk) {
    ChunkPlan p;
    p.seg_len = L;
    if (L <= 0 || batch <= 0 || D <= 0) return p;
    if (chunk > 0) {
        p.seg_len = chunk < L ? chunk : L;
    } else {
        const int64_t channels = batch * D;
        const bool filled = channels >= 8192 && D % jscan::rows::kCh == 0;
        int64_t n = (filled || channels >= kSegLanes) ? 1 : kSegLanes / channels;
        const int64_t by_length = L / 256 > 1 ? L / 256 : 1;
        if (n > by_length) n = by_length;
        p.seg_len = (L + n - 1) / n;
        p.seg_len = (p.seg_len + 63) / 64 * 64;
        if (p.seg_len > L) p.seg_len = L;
    }
    p.n_seg = (L + p.seg_len - 1) / p.seg_len;
    return p;
}

// Whether the plan's grids fit the launchers: segment rows and scan work-groups, the carry
// pass's work-groups of carry::kPairs (channel, state) pairs, and 32-bit token indexes.
inline bool chunk_grids_fit(int64_t batch, int64_t D, const ChunkPlan &p) {
    return batch * p.n_seg <= (1 << 24) && batch * p.n_seg * ((D + 63) / 64) <= kMaxBlocks &&
           batch * D * JSCAN_D_STATE / jscan::carry::kPairs <= kMaxBlocks && p.seg_len < ((int64_t)1 << 31);
}

// Workspace bytes of a plan: h_loc / h_in [batch * n_seg][D][N] and delta sums [batch * n_seg][D].
inline int64_t chunk_workspace_bytes(const ChunkPlan &p, int64_t batch, int64_t D) {
    if (p.n_seg <= 1) return 0;
    return batch * p.n_seg * D * (JSCAN_D_STATE + 1) * 4;
}

}  // namespace host
}  // namespace jscan

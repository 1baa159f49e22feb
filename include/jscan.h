/*
 * jscan.h - C ABI of libjscan, the Mamba-1 (S6) selective state-space scan on AMD
 * Instinct MI355X (gfx950).
 *
 * The operation.  For every batch row b, channel d < D and state n < N = 16, the scan
 * runs the selective recurrence of the Jamba notes page ("Jamba: A Hybrid
 * Transformer-Mamba Language Model", section "Mamba layer", the S6 equation):
 *
 *     h_t[d,n] = exp(delta_t[d] * A[d,n]) * h_{t-1}[d,n] + (delta_t[d] * x_t[d]) * B_t[n]
 *     y_t[d]   = sum_n C_t[n] * h_t[d,n]
 *
 * The decay exp(delta A) and the input term delta B x are the discretised A-bar and
 * B-bar x of that equation.  delta, B and C are inputs that depend on the token (same
 * section).  A is real and diagonal, one value per (channel, state) (lesson page
 * "Jamba - Hybrid SSM-Transformer", section "Mamba-3", item 2).  d_state is 16 (notes
 * page, "Mamba layer").  Only h_{t-1} and the current token are needed to advance one
 * token, so decoding runs in constant memory (lesson page, section "SSM on one page").
 *
 * Arithmetic.  The state is fp32 and is never rounded to the input dtype.  Every state
 * element is advanced by the same fp32 expression in every entry point:
 *     h = fmaf(exp2(delta * A2), h, (delta * x) * B),   with A2 = A * log2(e) in fp32,
 * and exp2 is the hardware v_exp_f32.  Tokens are visited in increasing t, one after the
 * other.  So the state that jscan_prefill returns is bit-identical to the state after L
 * calls of jscan_step on the same tokens, starting from +0.0.  y accumulates in fp32 and is
 * rounded to nearest even to the output dtype.  With bf16 output the prefill's sum over the
 * states runs on the matrix cores: its terms are rounded to bf16 once (2^-8 relative) and
 * summed in fp32 (the products C_t[n] h_t[d,n] with h rounded, or, in jscan_prefill_fused, the
 * lanes' fp32 partial sums over two states).  A NaN in a channel's state then also reaches
 * that channel's outputs earlier in the same 16-token group (a NaN term times a zero weight of
 * the summing matrix), never another channel.
 *
 * Layouts.  All arrays are row-major with the last index contiguous:
 *     x, delta, y : [batch][L][D]      B, C : [batch][L][N]
 *     A           : [D][N] fp32        h0, h, h_final : [batch][D][N] fp32
 * x, delta, B, C and y share one dtype (jscan_dtype).
 *
 * Ownership and execution.  Every array pointer is a DEVICE pointer that the caller
 * allocates, owns and frees.  The library allocates no memory, keeps no state between
 * calls and never synchronises.  Work is enqueued on `stream` (a hipStream_t; NULL means
 * the default stream), and results are valid once that stream has been synchronised.
 * Calls on different streams may run from different host threads.
 *
 * Errors.  Arguments are checked before anything is launched.  On any error nothing is
 * launched and no output is touched.
 *     JSCAN_ERR_NULL   a required pointer is NULL
 *     JSCAN_ERR_SHAPE  negative sizes, N != 16, D not a multiple of 8, a row stride
 *                      shorter than its row or not a multiple of 8, D above 2^24 or batch
 *                      above 2^20 (the kernels index channels and rows in 32 bits)
 *     JSCAN_ERR_DTYPE  unknown dtype
 *     JSCAN_ERR_ALIGN  an array pointer not 16-byte aligned
 *     JSCAN_ERR_ALIAS  an output overlaps an input or another output (the exceptions are
 *                      the in-place state of jscan_step, and h0 == h_final exactly for
 *                      jscan_prefill_resume)
 *     JSCAN_ERR_HIP    the launch failed; jscan_last_hip_error() gives the hipError_t
 *     JSCAN_ERR_WORKSPACE  the workspace passed to jscan_prefill_chunked is too small
 *     JSCAN_ERR_FORM   unknown form of A (jscan_a_form)
 * Faults inside a kernel surface at the caller's next synchronisation.  A is not
 * range-checked.  With delta >= 0 and A <= 0 the decay lies in (0, 1] and the recurrence
 * is stable; other values may overflow.  Zero-sized work (batch == 0 or D == 0) returns
 * JSCAN_OK without touching anything.
 */
#ifndef JSCAN_H
#define JSCAN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    JSCAN_OK = 0,
    JSCAN_ERR_NULL = 1,
    JSCAN_ERR_SHAPE = 2,
    JSCAN_ERR_DTYPE = 3,
    JSCAN_ERR_ALIGN = 4,
    JSCAN_ERR_ALIAS = 5,
    JSCAN_ERR_HIP = 6,
    JSCAN_ERR_WORKSPACE = 7,
    JSCAN_ERR_FORM = 8
} jscan_status;

/* dtype of x, delta, B, C and y.  A and every state are always fp32. */
typedef enum { JSCAN_F32 = 0, JSCAN_BF16 = 1 } jscan_dtype;

#define JSCAN_D_STATE 16

/*
 * Prefill: scan L tokens from the zero state.  Writes y for every token and the state after
 * the last token.
 *   x, delta [batch][L][D]   inputs (delta is used as given: no softplus or bias is applied)
 *   A        [D][N]          fp32 diagonal of A
 *   B, C     [batch][L][N]   inputs
 *   y        [batch][L][D]   output, same dtype as x
 *   h_final  [batch][D][N]   output fp32 state after token L-1 (zeros when L == 0)
 * With L == 0, x, delta, B, C and y may be NULL.
 */
jscan_status jscan_prefill(const void *x, const void *delta, const float *A, const void *B,
                           const void *C, void *y, float *h_final, int64_t batch, int64_t L,
                           int64_t D, int64_t N, jscan_dtype dtype, void *stream);

/*
 * Prefill from a caller-supplied state h0 [batch][D][N] fp32 instead of zeros.  This resumes
 * a scan: scanning tokens [0, L1) and then resuming over [L1, L) gives bit-identical y and
 * h_final to one prefill over [0, L).  h0 may equal h_final (an in-place update of the
 * state) but must not partly overlap it.  The other arguments are as for jscan_prefill.
 */
jscan_status jscan_prefill_resume(const void *x, const void *delta, const float *A,
                                  const void *B, const void *C, const float *h0, void *y,
                                  float *h_final, int64_t batch, int64_t L, int64_t D,
                                  int64_t N, jscan_dtype dtype, void *stream);

/*
 * Time-parallel prefill, for shapes whose batch * D channels are too few to fill the GPU
 * (a single sequence of a channel-sharded layer, for example).  Same inputs and outputs as
 * jscan_prefill_resume (h0 may be NULL for the zero state, and may equal h_final), computed
 * in three passes over segments of `chunk` tokens:
 *   1. every segment is scanned from the zero state, giving its end state h_loc[s] and,
 *      per channel, the sum of its delta values S[s];
 *   2. the segments' starting states follow in order from h_in[0] = h0 by composing the
 *      per-segment maps: h_in[s+1] = exp(A * S[s]) * h_in[s] + h_loc[s];
 *   3. every segment is scanned again from h_in[s], writing y and (last segment) h_final.
 * Pass 2 rests on the recurrence being affine in h: over a run of tokens the map
 * h -> exp(delta A) h + delta B x composes to h -> exp(A * sum delta) h + h_loc, where h_loc
 * is the run's end state from zero (S6 equation, notes page "Jamba: A Hybrid
 * Transformer-Mamba Language Model", section "Mamba layer").
 * Rounding: with fp32 output the first segment's y is bit-identical to jscan_prefill_resume's
 * (with bf16 output it agrees to the rounding of the prefill's sum over states); later
 * segments start from composed states whose rounding differs from the token-by-token walk,
 * so their y and h_final agree with it to within fp32 rounding of the composition, not bit
 * for bit.  Results are deterministic (no atomics; fixed summation orders).
 *   chunk      tokens per segment; 0 picks enough segments for four waves per SIMD (262144
 *              segment-channel lanes, segments of at least 256 tokens), or one segment when
 *              batch * D already fills the GPU (at least 8192 channels, D a multiple of 32).  When it yields a
 *              single segment the call is exactly jscan_prefill_resume (and needs no
 *              workspace).
 *   workspace  device memory of at least jscan_prefill_chunked_workspace(...) bytes,
 *              16-byte aligned, owned by the caller, not overlapping any other array;
 *              may be NULL when that size is 0.  Its contents on entry do not matter.
 * Calls that share a workspace must be ordered on one stream.
 */
jscan_status jscan_prefill_chunked(const void *x, const void *delta, const float *A,
                                   const void *B, const void *C, const float *h0, void *y,
                                   float *h_final, int64_t batch, int64_t L, int64_t D,
                                   int64_t N, int64_t chunk, void *workspace,
                                   int64_t workspace_bytes, jscan_dtype dtype, void *stream);

/*
 * Workspace bytes jscan_prefill_chunked needs for this shape and chunk (0 when it runs as
 * a single segment), or -1 if the shape or chunk is invalid.  Host-only; launches nothing.
 */
int64_t jscan_prefill_chunked_workspace(int64_t batch, int64_t L, int64_t D, int64_t N,
                                        int64_t chunk);

/*
 * Producer side: the scan's delta, B and C computed from x (bf16 only), for M tokens.
 * The notes page ("Jamba: A Hybrid Transformer-Mamba Language Model", section "Mamba layer")
 * makes these parameters functions of the input and applies RMSNorm in the Mamba layer;
 * they are computed as the selective projection of Mamba-1:
 *     [d_low | B | C] = W_x x_t                          (fp32 accumulation of bf16 products)
 *     d_low = rmsnorm(d_low) * g_delta,  B = rmsnorm(B) * g_B,  C = rmsnorm(C) * g_C,
 *             rmsnorm(v) = v / sqrt(mean(v^2) + eps) over each vector's own width
 *     delta = softplus(W_dt d_low + b_dt)
 * Each output is rounded once, to nearest even, from its fp32 value.  The products run on the
 * matrix cores (MFMA 16x16x32 bf16); the normalisation, bias and softplus run on the fp32
 * accumulators before the rounding.
 *   x          [M][D]      bf16, M = batch * L tokens in any order (rows are independent)
 *   w_x        [R + 2N][D] bf16: rows 0..R-1 give d_low, R..R+N-1 give B, R+N.. give C
 *   g_delta [R], g_B [N], g_C [N]   fp32 gains
 *   w_dt       [D][R]      bf16 (row d produces channel d)
 *   b_dt       [D]         fp32
 *   delta_low  [M][R]      out, bf16, the normalised d_low (also the input of the second product)
 *   delta      [M][D]      out, bf16;   B, C [M][N] out, bf16
 * R must be 64, 128 or 256; N = 16; D a multiple of 128; 0 <= M <= 2^31; eps in [0, 1].  dtype must be
 * JSCAN_BF16 (JSCAN_ERR_DTYPE otherwise).  Outputs must not overlap inputs or each other.
 * Two kernels are launched on `stream`, in order.  With delta == NULL only the first
 * product runs (delta_low, B and C; w_dt and b_dt may then be NULL): the input of
 * jscan_prefill_fused, which computes delta itself.
 */
jscan_status jscan_ssm_inputs(const void *x, const void *w_x, const float *g_delta, const float *g_B,
                              const float *g_C, const void *w_dt, const float *b_dt, void *delta_low,
                              void *delta, void *B, void *C, int64_t M, int64_t D, int64_t R,
                              int64_t N, float eps, jscan_dtype dtype, void *stream);

/*
 * Prefill with the second product of jscan_ssm_inputs folded into the scan's load path: delta
 * is never stored.  The kernel computes, tile by tile, delta = softplus(W_dt delta_low + b_dt)
 * with the same matrix-core sequence, bias add, softplus and bf16 rounding as
 * jscan_ssm_inputs, so h_final is bit-identical to jscan_ssm_inputs followed by
 * jscan_prefill_resume (jscan_prefill when h0 is NULL).  y agrees with it to the rounding of the
 * sum over states: this kernel's matrix cores also compute delta, so it sums the lanes' partials
 * there (half the MFMAs) rather than contracting the states with C.
 *   x          [batch][L][D] bf16      delta_low [batch][L][R] bf16 (from jscan_ssm_inputs)
 *   w_dt       [D][R] bf16             b_dt [D] fp32
 *   A, B, C, h0 (may be NULL), y, h_final as for jscan_prefill_resume
 * Limits: bf16 only, R = 256, D a multiple of 32 (the shapes of the row-mapped prefill);
 * other shapes return JSCAN_ERR_SHAPE and are served by jscan_ssm_inputs then jscan_prefill.
 */
jscan_status jscan_prefill_fused(const void *x, const void *delta_low, const void *w_dt,
                                 const float *b_dt, const float *A, const void *B, const void *C,
                                 const float *h0, void *y, float *h_final, int64_t batch,
                                 int64_t L, int64_t D, int64_t N, int64_t R, jscan_dtype dtype,
                                 void *stream);

/*
 * Decode step: advance the state by one token, in place, and write that token's output.
 *   h        [batch][D][N] fp32, read and overwritten with the new state
 *   x_t, delta_t: batch rows of D values; row b starts at element b * ld_xd
 *   A        [D][N] fp32
 *   B_t, C_t: batch rows of N values; row b starts at element b * ld_bc
 *   y_t      batch rows of D values; row b starts at element b * ld_y; same dtype as x_t
 * The strides let a caller pass token t of prefill-layout tensors without a copy
 * (x + t*D with ld_xd = L*D, B + t*N with ld_bc = L*N), and write y_t either into a
 * prefill-layout output (y + t*D with ld_y = L*D) or into a contiguous [batch][D] (ld_y = D).
 * ld_xd >= D, ld_bc >= N, ld_y >= D, and all three must be multiples of 8.
 */
jscan_status jscan_step(float *h, const void *x_t, const void *delta_t, const float *A,
                        const void *B_t, const void *C_t, void *y_t, int64_t batch, int64_t D,
                        int64_t N, int64_t ld_xd, int64_t ld_bc, int64_t ld_y, jscan_dtype dtype,
                        void *stream);

/*
 * Scaled-identity A (the Mamba-2 form).  The lesson page ("Jamba - Hybrid SSM-Transformer",
 * section "Mamba-3", item 2) describes Mamba-2's state matrix as a scaled identity instead of
 * Mamba-1's real diagonal; everything else about the layer is taken to be unchanged (same
 * Euler-style input term, same delta, B, C and y).  So A is one value per channel:
 *     A[d][n] = a[d] for every n,   a [D] fp32.
 * The decay exp(delta_t[d] * a[d]) is then the same for all 16 states of a channel, and these
 * kernels evaluate it once per (token, channel) instead of once per state element, by the
 * same fp32 expression as the general kernels.  Their y, h_final and decode states are
 * therefore bit-identical to jscan_prefill_resume / jscan_step run on the expanded A[d][n] =
 * a[d], only faster.
 *
 * Prefill from h0 (NULL for the zero state; h0 may equal h_final).  The other arguments,
 * layouts and errors are those of jscan_prefill_resume, with `a` [D] fp32 in place of A.
 */
jscan_status jscan_prefill_scalar_a(const void *x, const void *delta, const float *a,
                                    const void *B, const void *C, const float *h0, void *y,
                                    float *h_final, int64_t batch, int64_t L, int64_t D,
                                    int64_t N, jscan_dtype dtype, void *stream);

/* Decode step with a scaled-identity A: jscan_step with `a` [D] fp32 in place of A. */
jscan_status jscan_step_scalar_a(float *h, const void *x_t, const void *delta_t, const float *a,
                                 const void *B_t, const void *C_t, void *y_t, int64_t batch,
                                 int64_t D, int64_t N, int64_t ld_xd, int64_t ld_bc,
                                 int64_t ld_y, jscan_dtype dtype, void *stream);

/*
 * Complex-valued state (the Mamba-3 form).  The lesson page ("Jamba - Hybrid SSM-Transformer",
 * section "Mamba-3", item 2) has Mamba-3 bring back a complex state matrix, which amounts to
 * multiplying the state by a data-dependent rotation.  Here the 16 real state components of a
 * channel are read as 8 complex states, h[k] = h[2k] + i h[2k+1], and A[d][2k], A[d][2k+1] as
 * the real and imaginary parts of its complex diagonal entry a; B and C pair up the same way.
 * The S6 equation in complex arithmetic then reads
 *     h_t[k] = exp(delta_t a) h_{t-1}[k] + (delta_t x_t) (B_t[2k] + i B_t[2k+1])
 *     y_t    = sum_n C_t[n] h_t[n]            (= sum_k Re(conj(c_k) h_t[k]))
 * with exp(delta a) = 2^(delta Re(a) log2 e) (cos(delta Im a) + i sin(delta Im a)): a decay by
 * the real part and a rotation by the imaginary part.  With every Im a = 0 this is the real
 * diagonal scan with A[d][2k+1] = A[d][2k].  Every entry point advances the pairs with the same
 * fp32 expression (hardware sine and cosine of the angle in turns, reduced to [0, 1)), so the
 * prefill's final state equals the step chain's bit for bit.  States, h0 and h_final keep the
 * [batch][D][16] fp32 layout with the pairs interleaved.  Re(a) <= 0 keeps the recurrence
 * stable; Im(a) is an angle rate in radians per unit of delta.  The other arguments, layouts
 * and errors are those of jscan_prefill_resume (h0 may be NULL) and jscan_step.
 */
jscan_status jscan_prefill_complex(const void *x, const void *delta, const float *A,
                                   const void *B, const void *C, const float *h0, void *y,
                                   float *h_final, int64_t batch, int64_t L, int64_t D,
                                   int64_t N, jscan_dtype dtype, void *stream);

/* Decode step with the complex-valued state (see jscan_prefill_complex). */
jscan_status jscan_step_complex(float *h, const void *x_t, const void *delta_t, const float *A,
                                const void *B_t, const void *C_t, void *y_t, int64_t batch,
                                int64_t D, int64_t N, int64_t ld_xd, int64_t ld_bc,
                                int64_t ld_y, jscan_dtype dtype, void *stream);

/*
 * Exponential-trapezoidal discretisation, the Mamba-3 replacement of the Euler rule (lesson
 * page "Jamba - Hybrid SSM-Transformer", section "Mamba-3", item 1: the input term of the
 * recurrence mixes neighbouring tokens).  The input integral over step t is weighted lam_t at
 * the step's right end (this token) and 1 - lam_t at its left end (the previous token), which
 * decays with the state over the step:
 *
 *     h_t = exp(delta_t a) (h_{t-1} + ((1 - lam_t) delta_t) x_{t-1} B_{t-1}) + ((lam_t delta_t) x_t) B_t
 *
 * in fp32 as k = fmaf(p, B_{t-1}, h), p = ((1 - lam) * delta) * x_{t-1}, then the form's usual
 * update of k with q = (lam * delta) * x_t in place of delta * x_t.  y_t = C_t h_t as before.
 * lam = 1 is the Euler rule of the other entry points, bit for bit.  lam_t in [0, 1] is
 * expected (not checked).  The rule combines with every form of A:
 *     JSCAN_A_DIAGONAL         A [D][N]: the Mamba-1 form of jscan_prefill
 *     JSCAN_A_SCALED_IDENTITY  a [D]: the Mamba-2 form of jscan_prefill_scalar_a
 *     JSCAN_A_COMPLEX          A [D][N] as (real, imaginary) pairs: jscan_prefill_complex
 */
typedef enum { JSCAN_A_DIAGONAL = 0, JSCAN_A_SCALED_IDENTITY = 1, JSCAN_A_COMPLEX = 2 } jscan_a_form;

/*
 * Prefill with the exponential-trapezoidal rule, from h0 (NULL: zero state).
 *   lam     [batch][L][D], the dtype of x: the right-end weight of each (token, channel).
 *   x_prev  [batch][D] and B_prev [batch][N], the dtype of x: the token before the first one,
 *           whose input is the first step's left end point.  Both NULL when the sequence
 *           starts here (that term is then zero); a resumed sequence passes its last token.
 * Other arguments, layouts, errors and the bit-identity of h_final with the step chain are
 * as for jscan_prefill_resume (with jscan_step_trapezoid as the step).  Added errors:
 * JSCAN_ERR_NULL when lam is NULL or only one of x_prev and B_prev is, JSCAN_ERR_FORM for an
 * unknown a_form, JSCAN_ERR_ALIAS when y or h_final overlaps lam, x_prev or B_prev.
 */
jscan_status jscan_prefill_trapezoid(const void *x, const void *delta, const void *lam, const float *A,
                                     const void *B, const void *C, const float *h0, const void *x_prev,
                                     const void *B_prev, void *y, float *h_final, int64_t batch, int64_t L,
                                     int64_t D, int64_t N, jscan_a_form a_form, jscan_dtype dtype,
                                     void *stream);

/*
 * Decode step with the exponential-trapezoidal rule.  x_prev (rows of D, stride ld_xd) and
 * B_prev (rows of N, stride ld_bc) are the previous token's x and B, required: zeros for a
 * sequence's first token.  lam_t has the rows of x_t.  Otherwise as jscan_step (h in place).
 */
jscan_status jscan_step_trapezoid(float *h, const void *x_prev, const void *B_prev, const void *x_t,
                                  const void *delta_t, const void *lam_t, const float *A, const void *B_t,
                                  const void *C_t, void *y_t, int64_t batch, int64_t D, int64_t N,
                                  int64_t ld_xd, int64_t ld_bc, int64_t ld_y, jscan_a_form a_form,
                                  jscan_dtype dtype, void *stream);

/*
 * Multi-input, multi-output (MIMO) scan, the Mamba-3 replacement of the per-channel scalar
 * projections by matrix-valued ones (lesson page "Jamba - Hybrid SSM-Transformer", section
 * "Mamba-3", item 3).  Each channel takes R inputs and gives R outputs; B_t and C_t are N x R
 * matrices shared by the channels; the state keeps its [batch][D][N] size:
 *
 *     h_t[d][n] = exp(delta_t[d] a) h_{t-1}[d][n] + sum_r (delta_t[d] * x_t[d][r]) * B_t[n][r]
 *     y_t[d][r] = sum_n C_t[n][r] * h_t[d][n]
 *
 * with the sum over r accumulated in increasing r (first product, then fmaf), and the decay a
 * of any form of A (jscan_a_form; with JSCAN_A_COMPLEX the state pairs, and B's and C's row
 * pairs for each r, are complex numbers).  R = 1 is the single-input scan of the form's
 * entry point, bit for bit in the state.  R must be 1, 2, 4 or 8 (else JSCAN_ERR_SHAPE).
 *
 * Prefill from h0 (NULL: zero state).  Layouts:
 *     x, y : [batch][L][D][R]     delta : [batch][L][D]     B, C : [batch][L][N][R]
 * Other arguments, ownership, errors (plus JSCAN_ERR_FORM) and the bit-identity of h_final
 * with the jscan_step_mimo chain are as for jscan_prefill_resume.
 */
jscan_status jscan_prefill_mimo(const void *x, const void *delta, const float *A, const void *B,
                                const void *C, const float *h0, void *y, float *h_final,
                                int64_t batch, int64_t L, int64_t D, int64_t N, int64_t R,
                                jscan_a_form a_form, jscan_dtype dtype, void *stream);

/*
 * One MIMO decode token for a batch, h [batch][D][N] in place.  x_t is rows of D * R with
 * row stride ld_x; delta_t rows of D with stride ld_d; B_t and C_t rows of N * R with stride
 * ld_bc; y_t rows of D * R with stride ld_y (strides in elements, multiples of 8, at least the
 * row length).
 */
jscan_status jscan_step_mimo(float *h, const void *x_t, const void *delta_t, const float *A,
                             const void *B_t, const void *C_t, void *y_t, int64_t batch, int64_t D,
                             int64_t N, int64_t R, int64_t ld_x, int64_t ld_d, int64_t ld_bc,
                             int64_t ld_y, jscan_a_form a_form, jscan_dtype dtype, void *stream);

/*
 * The MIMO scan with the exponential-trapezoidal rule: both Mamba-3 changes together.  The
 * rank-R input u_t[n] = sum_r x_t[d][r] B_t[n][r] takes the place of x_t B_t at both end
 * points of the step, in fp32 as
 *     k = h;  k = fmaf(p_r, B_{t-1}[n][r], k) for r = 0 .. R-1,   p_r = ((1 - lam) * delta) * x_{t-1}[d][r]
 * then the MIMO update of k with q_r = (lam * delta) * x_t[d][r] in place of delta * x_t[d][r].
 * lam = 1 is jscan_prefill_mimo bit for bit; R = 1 is jscan_prefill_trapezoid bit for bit.
 * lam [batch][L][D] (delta's layout); x_prev [batch][D][R] and B_prev [batch][N][R] are the token
 * before the first (both NULL when there is none).  Other arguments, layouts and errors as for
 * jscan_prefill_mimo and jscan_prefill_trapezoid.
 */
jscan_status jscan_prefill_mimo_trapezoid(const void *x, const void *delta, const void *lam,
                                          const float *A, const void *B, const void *C,
                                          const float *h0, const void *x_prev, const void *B_prev,
                                          void *y, float *h_final, int64_t batch, int64_t L,
                                          int64_t D, int64_t N, int64_t R, jscan_a_form a_form,
                                          jscan_dtype dtype, void *stream);

/*
 * One MIMO decode token with the exponential-trapezoidal rule.  x_prev has x_t's rows (stride
 * ld_x), B_prev B_t's (ld_bc), lam_t delta_t's (ld_d); all three required (zeros before a
 * sequence's first token).  Otherwise as jscan_step_mimo.
 */
jscan_status jscan_step_mimo_trapezoid(float *h, const void *x_prev, const void *B_prev,
                                       const void *x_t, const void *delta_t, const void *lam_t,
                                       const float *A, const void *B_t, const void *C_t, void *y_t,
                                       int64_t batch, int64_t D, int64_t N, int64_t R, int64_t ld_x,
                                       int64_t ld_d, int64_t ld_bc, int64_t ld_y,
                                       jscan_a_form a_form, jscan_dtype dtype, void *stream);

/*
 * jscan_prefill_chunked without a workspace argument, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc).  It runs the same three passes on the same kernels, with the segment states and
 * delta sums in a library-owned scratch array of JSCAN_NOALLOC_SCRATCH_BYTES in each GPU's
 * memory (a static device array, held until the process ends).  The call itself allocates
 * nothing; the first call on a device looks up that device's copy of the array once.
 *   - A shape and chunk whose jscan_prefill_chunked_workspace(...) exceeds
 *     JSCAN_NOALLOC_SCRATCH_BYTES returns JSCAN_ERR_WORKSPACE and launches nothing (24 MiB
 *     holds every automatic plan, which needs at most 262144 * 68 bytes = 17 MiB; explicit
 *     chunks need batch * n_seg * D * 68 bytes).
 *   - Every call on one GPU uses that GPU's one array: calls that overlap in time on one GPU
 *     (from different streams or threads, or an unordered graph) race and give wrong results.
 *     Order them on one stream.  The array's contents on entry do not matter (every element
 *     the passes read was written earlier in the same call).
 * The other arguments, the results and the errors are those of jscan_prefill_chunked; a
 * failure to look up the array returns JSCAN_ERR_HIP.
 */
#define JSCAN_NOALLOC_SCRATCH_BYTES (24 * 1024 * 1024)
jscan_status jscan_prefill_chunked_noalloc(const void *x, const void *delta, const float *A,
                                           const void *B, const void *C, const float *h0, void *y,
                                           float *h_final, int64_t batch, int64_t L, int64_t D,
                                           int64_t N, int64_t chunk, jscan_dtype dtype, void *stream);

/*
 * Gated recurrence: the linear recurrence without the expansion over d_state, its gate an input.
 * One fp32 state per (sequence, channel):
 *     JSCAN_GATE_DECAY     h_t = exp(g_t) h_{t-1} + u_t                          (g a log decay)
 *     JSCAN_GATE_SIGMOID   h_t = sigmoid(g_t) h_{t-1} + (1 - sigmoid(g_t)) u_t   (g a gate logit)
 *     y_t = h_t, rounded to nearest even to the dtype
 * g = -inf makes the decay 0, which drops a finite state before the token (a reset inside a row).  It is a
 * product like any other: 0 times an infinity or a NaN is NaN, so a reset does not clear those (nor
 * do decays whose product underflows to 0).  They stay in their channel to the end of their sequence,
 * in the backward pass (from dy) to its start, and reach no other channel or sequence.  Documents that
 * must not reach each other in that case are sequences of their own.  Gates that make the recurrence
 * unstable (g > 0 in the decay form) are not checked; the decays of any run of tokens have to multiply to
 * a finite fp32 number.
 *
 * Scan over whole sequences.
 *   g, u, y   batch * L token rows of D values in `dtype`; the row of token t of sequence b starts at
 *             element (b * L + t) * ld (ld_g, ld_u, ld_y >= D).  So g and u may be the halves of one
 *             [batch][L][2 D] projection.  Any D >= 0 and any ld; tensors whose rows all start on 4 bytes
 *             (bf16: even D, ld and start) run faster.  Pointers are aligned to their elements.
 *   h0        [batch][D] fp32 state before the first token, or NULL for zeros; may equal h_final
 *   lengths   [batch] int32 in device memory, or NULL when every sequence has L tokens.  Sequence b
 *             has lengths[b] tokens (taken into [0, L]); its later rows of g and u are not read, and
 *             its later rows of y are set to zero
 *   h_final   [batch][D] fp32 state after the last token (h0 for an empty sequence)
 *   workspace device memory of jscan_gated_scan_workspace(batch, L, D) bytes, 16-byte aligned,
 *             overlapping nothing else; may be NULL when that is 0.  Contents on entry do not
 *             matter.  Calls that share a workspace must be ordered on one stream.
 * A long axis is cut into segments that run side by side and are joined through their composed
 * maps, so states agree with the decode-step chain to the fp32 rounding of that composition, not
 * bit for bit.  Results are deterministic (fixed orders, no atomics).  With L == 0, g, u and y may
 * be NULL.  Errors as for jscan_prefill_chunked, and JSCAN_ERR_FORM for an unknown form.
 */
typedef enum { JSCAN_GATE_DECAY = 0, JSCAN_GATE_SIGMOID = 1 } jscan_gate_form;

jscan_status jscan_gated_scan(const void *g, const void *u, const float *h0, const int32_t *lengths,
                              void *y, float *h_final, int64_t batch, int64_t L, int64_t D,
                              int64_t ld_g, int64_t ld_u, int64_t ld_y, void *workspace,
                              int64_t workspace_bytes, jscan_gate_form form, jscan_dtype dtype,
                              void *stream);

/* Workspace bytes of jscan_gated_scan and jscan_gated_scan_backward for this shape (the same for
 * both, either form, either dtype), or -1 if the shape is invalid.  Host-only. */
int64_t jscan_gated_scan_workspace(int64_t batch, int64_t L, int64_t D);

/*
 * Backward pass of jscan_gated_scan.  With G_t = dLoss/dh_t, c_t = a_t G_t and a_t the decay:
 *     G_t = dy_t + c_{t+1}   (dh_final in place of c after the last token),   dh0 = c_1
 *     JSCAN_GATE_DECAY     du_t = G_t               dg_t = c_t h_{t-1}
 *     JSCAN_GATE_SIGMOID   du_t = (1 - a_t) G_t     dg_t = c_t (1 - a_t) (h_{t-1} - u_t)
 * G and c are fp32; h_{t-1} is read from y, so for bf16 dg carries y's one rounding: an error of at most
 * 2^-8 |c_t h_{t-1}| in the decay form and 2^-8 |c_t (1 - a_t) h_{t-1}| in the sigmoid form, where
 * h_{t-1} - u_t may cancel, so that it has no bound relative to dg (10% and more where states and
 * inputs are close).  jscan_gated_scan_backward_saved, below, has h in fp32.
 *   g, u, y, dy   token rows as above; u may be NULL (and is not read) in the decay form; y is the
 *                 scan's output
 *   h0            the scan's, NULL for zeros;   dh_final [batch][D] fp32, NULL for zeros
 *   lengths       as for the scan; rows of padding are not read
 *   dg, du        token rows out, in `dtype`; zero in rows of padding.  They may be the halves of one
 *                 [batch][L][2 D] buffer
 *   dh0           [batch][D] fp32 out, or NULL when it is not wanted; may equal dh_final
 * Workspace, errors and determinism as for jscan_gated_scan.
 */
jscan_status jscan_gated_scan_backward(const void *g, const void *u, const void *y, const void *dy,
                                       const float *h0, const float *dh_final,
                                       const int32_t *lengths, void *dg, void *du, float *dh0,
                                       int64_t batch, int64_t L, int64_t D, int64_t ld_g,
                                       int64_t ld_u, int64_t ld_y, int64_t ld_dy, int64_t ld_dg,
                                       int64_t ld_du, void *workspace, int64_t workspace_bytes,
                                       jscan_gate_form form, jscan_dtype dtype, void *stream);

/*
 * Training in bf16 with fp32 states.  jscan_gated_scan_save is jscan_gated_scan that also keeps the fp32 state
 * before every eighth token; jscan_gated_scan_backward_saved is jscan_gated_scan_backward that walks up from
 * them, so that no h is rounded to bf16 (y and h0 are not needed; u is, in both forms).
 *   states    [batch][ceil(L / 8)][D] fp32, jscan_gated_scan_states(batch, L, D) bytes, 16-byte aligned: row r
 *             of a sequence is its state before token 8 r.  Rows behind a sequence's last token are
 *             neither written nor read
 * JSCAN_BF16 only (JSCAN_ERR_DTYPE otherwise): with JSCAN_F32 y itself holds the states.  With L == 0,
 * states may be NULL.  Everything else as for the calls without it; y, h_final, du and dh0 agree with
 * theirs to the fp32 rounding of the composition.
 */
jscan_status jscan_gated_scan_save(const void *g, const void *u, const float *h0,
                                   const int32_t *lengths, void *y, float *h_final, float *states,
                                   int64_t batch, int64_t L, int64_t D, int64_t ld_g, int64_t ld_u,
                                   int64_t ld_y, void *workspace, int64_t workspace_bytes,
                                   jscan_gate_form form, jscan_dtype dtype, void *stream);

/* Bytes of states for this shape, or -1 if the shape is invalid.  Host-only. */
int64_t jscan_gated_scan_states(int64_t batch, int64_t L, int64_t D);

jscan_status jscan_gated_scan_backward_saved(const void *g, const void *u, const float *states,
                                             const void *dy, const float *dh_final,
                                             const int32_t *lengths, void *dg, void *du, float *dh0,
                                             int64_t batch, int64_t L, int64_t D, int64_t ld_g,
                                             int64_t ld_u, int64_t ld_dy, int64_t ld_dg,
                                             int64_t ld_du, void *workspace,
                                             int64_t workspace_bytes, jscan_gate_form form,
                                             jscan_dtype dtype, void *stream);

/*
 * One decode token of the gated recurrence for a batch: h [batch][D] fp32 in place; g_t, u_t and y_t
 * are batch rows of D values with row strides ld_g, ld_u, ld_y >= D.
 */
jscan_status jscan_gated_step(float *h, const void *g_t, const void *u_t, void *y_t, int64_t batch,
                              int64_t D, int64_t ld_g, int64_t ld_u, int64_t ld_y,
                              jscan_gate_form form, jscan_dtype dtype, void *stream);

/*
 * A linear layer with weights and activations in 8-bit integers (the review page of Jamba-1.5,
 * section 3-2.3, holds the model's expert weights in int8 for serving).
 *
 * Row quantiser: every row (token) of x gets a scale of its own,
 *     scale[m] = max(max_k |x[m][k]| * (1 / 127), 2^-126),   q[m][k] = rint(x[m][k] * (1 / scale[m]))
 * in fp32 (each bracket rounded first), ties to even.  A row that holds a NaN or an infinity gets scale NaN and q = 0, so the
 * product's row is NaN and no other row is touched.
 *   x      M rows of K values in `dtype`, row stride ld_x >= K elements; rows that start on 16 bytes
 *          run faster
 *   q      [M][K] int8 out, 16-byte aligned;   scale [M] fp32 out
 * K a multiple of 16, 16 <= K <= 131056; 0 <= M <= 2^30.
 */
jscan_status jscan_quantize_rows(const void *x, int8_t *q, float *scale, int64_t M, int64_t K,
                                 int64_t ld_x, jscan_dtype dtype, void *stream);

/*
 * Product with int8 weights, a scale for each token (row of q) and each output channel (row of w):
 *     out[m][n] = (sum_k q[m][k] w[n][k]) * q_scale[m] * w_scale[n] + bias[n]
 * The sum is int32 on the matrix cores and exact; scales and bias are applied in fp32 and the result
 * is rounded once to `dtype`.
 *   q [M][K], w [N][K]   int8, 16-byte aligned;   q_scale [M], w_scale [N] fp32
 *   bias                 [N] fp32 or NULL
 *   out                  M rows of N values in `dtype`, row stride ld_out >= N elements
 * K a multiple of 16, 16 <= K <= 131056; 0 <= M <= 2^30; 0 <= N <= 2^24; products
 * of more results than the tiles' grids count (about 2^38) are JSCAN_ERR_SHAPE.
 */
jscan_status jscan_matmul_i8(const int8_t *q, const float *q_scale, const int8_t *w,
                             const float *w_scale, const float *bias, void *out, int64_t M, int64_t N,
                             int64_t K, int64_t ld_out, jscan_dtype dtype, void *stream);

/*
 * Activations of the calls below, applied in fp32 before a result is rounded:
 *     JSCAN_ACT_SILU        v sigmoid(v)
 *     JSCAN_ACT_GELU_TANH   v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2
 */
typedef enum { JSCAN_ACT_NONE = 0, JSCAN_ACT_SILU = 1, JSCAN_ACT_GELU_TANH = 2 } jscan_activation;

/*
 * Short causal convolution in front of a scan: every channel over its own last W tokens (W = 2, 3 or 4).
 *     y_t[d] = act(bias[d] + sum_{k < W} w[d][k] e_{t+k}[d])
 * with e the W - 1 tokens of `state` followed by x_0, x_1, ..., so w[d][W-1] weighs the token itself.  Sums are
 * fp32.  act is JSCAN_ACT_NONE or JSCAN_ACT_SILU (JSCAN_ERR_FORM otherwise).
 *   x, y       batch * L token rows of D values in `dtype`, row strides ld_x, ld_y >= D as for
 *              jscan_gated_scan: x may be a half of a wider projection.  Any D >= 0; pointers are aligned to their
 *              elements
 *   state      [batch][W-1][D] in `dtype`, the tokens before the first (oldest first), or NULL for zeros
 *   w, bias    [D][W] and [D] fp32; bias may be NULL
 *   lengths    [batch] int32 or NULL, as for jscan_gated_scan: later rows of x are not read, later rows of y are
 *              set to zero (a selective scan behind this call takes no lengths: see jscan_prefill_gate)
 *   state_out  [batch][W-1][D] out, the last W - 1 tokens of every sequence (the starting state's among them where
 *              it is shorter), or NULL when it is not wanted; may equal state
 * With L == 0, x and y may be NULL.  Errors as above.
 */
jscan_status jscan_causal_conv(const void *x, const void *state, const float *w, const float *bias,
                               const int32_t *lengths, void *y, void *state_out, int64_t batch,
                               int64_t L, int64_t D, int64_t W, int64_t ld_x, int64_t ld_y,
                               jscan_activation activation, jscan_dtype dtype, void *stream);

/*
 * Backward pass of jscan_causal_conv.  With z_t = dy_t act'(v_t), v_t the sum that the activation takes,
 *     de_i = sum_k w[k] z_{i-k}  (and dstate_out's rows at the places that state_out was taken from)
 *     dw[d][k] = sum_t z_t e_{t+k},   dbias[d] = sum_t z_t       over all tokens of all sequences
 * v is formed anew from x, in fp32; z is not rounded; every sum is fp32, in a fixed order (no atomics).
 *   x, state, w, bias, lengths   as given to the forward pass
 *   dy          token rows like x;   dstate_out [batch][W-1][D] in `dtype`, NULL for zeros
 *   dx          token rows out, zero in the padding;   dstate [batch][W-1][D] out, NULL when it is not wanted
 *   dw, dbias   [D][W] and [D] fp32 out; dbias may be NULL
 *   workspace   jscan_causal_conv_backward_workspace(batch, L, D, W) bytes, 16-byte aligned, overlapping nothing
 *               else.  Contents on entry do not matter.  Calls that share it must be ordered on one stream.
 * Without any sequence (batch == 0) dw and dbias are set to zeros.
 */
jscan_status jscan_causal_conv_backward(const void *x, const void *state, const float *w,
                                        const float *bias, const int32_t *lengths, const void *dy,
                                        const void *dstate_out, void *dx, void *dstate, float *dw,
                                        float *dbias, int64_t batch, int64_t L, int64_t D, int64_t W,
                                        int64_t ld_x, int64_t ld_dy, int64_t ld_dx, void *workspace,
                                        int64_t workspace_bytes, jscan_activation activation,
                                        jscan_dtype dtype, void *stream);

/* Workspace bytes of jscan_causal_conv_backward for this shape, or -1 if the shape is invalid.  Host-only. */
int64_t jscan_causal_conv_backward_workspace(int64_t batch, int64_t L, int64_t D, int64_t W);

/*
 * One decode token of the convolution for a batch: state [batch][W-1][D] in place (its oldest token leaves, x_t
 * joins); x_t and y_t are batch rows of D values with row strides ld_x, ld_y >= D.
 */
jscan_status jscan_causal_conv_step(void *state, const void *x_t, const float *w, const float *bias,
                                    void *y_t, int64_t batch, int64_t D, int64_t W, int64_t ld_x,
                                    int64_t ld_y, jscan_activation activation, jscan_dtype dtype,
                                    void *stream);

/*
 * The selective scan with what follows it in its layer, the skip and the output gate, in one pass:
 *     y_t[d] = (sum_n C_t[n] h_t[d,n] + skip[d] x_t[d]) silu(z_t[d])
 * rounded once from fp32.  skip or z may be NULL (its part is left out; not both).  h is the scan's, bit for bit (see chunk).
 * The sum over n is fp32, but for one case that the caller chooses by chunk: with bf16 and D a multiple of 32 a
 * token-by-token call (chunk -1, or any call with another a_form) forms it as jscan_prefill does, each state rounded to
 * bf16 on its way into the sum (see Arithmetic above).  What enters the skip and the gate is then off by up to
 * 2^-8 sum_n |C_t[n] h_t[d,n]|, which stays where C h and skip x cancel, and a NaN reaches earlier tokens of its channel.
 *   skip      [D] fp32
 *   z         batch * L token rows of D values in `dtype`, row stride ld_z >= D (a multiple of 8, at most 2^25), in the
 *             order of x's rows: z may be a half of a wider projection
 *   chunk     -1: token by token (h is jscan_prefill_resume's, or that of a_form's prefill); above 0: in segments
 *             of that many tokens (h is jscan_prefill_chunked's); 0: whichever way is expected to be fastest for this
 *             shape among those that sum in fp32.  Segments are for JSCAN_A_DIAGONAL: for the other forms 0 is token
 *             by token and a given length is JSCAN_ERR_FORM
 *   workspace jscan_prefill_gate_workspace(batch, L, D, N, chunk) bytes where a_form is JSCAN_A_DIAGONAL; else, and
 *             where that is 0, it may be NULL
 *   h0        [batch][D][N] fp32 or NULL for zeros; may equal h_final
 * There are no lengths.  In a padded batch the caller sets delta to zero behind every sequence, where x, B and C must be
 * finite (jscan_causal_conv leaves zeros there; a delta projected from them is not zero): such a token leaves the
 * state as it is.  y's rows there are not zero.
 * The other arguments and the errors are those of jscan_prefill_chunked.
 */
jscan_status jscan_prefill_gate(const void *x, const void *delta, const float *A, const void *B,
                                const void *C, const float *h0, const float *skip, const void *z,
                                void *y, float *h_final, int64_t batch, int64_t L, int64_t D, int64_t N,
                                int64_t ld_z, int64_t chunk, void *workspace, int64_t workspace_bytes,
                                jscan_a_form a_form, jscan_dtype dtype, void *stream);

/* Workspace bytes of jscan_prefill_gate for this shape, or -1 if the shape or chunk is invalid.  Host-only. */
int64_t jscan_prefill_gate_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t chunk);

/*
 * One decode token of it for a batch: jscan_step (or the step of a_form) with the skip and the gate.  z_t's rows
 * have the stride ld_z >= D (a multiple of 8, at most 2^25).
 */
jscan_status jscan_step_gate(float *h, const void *x_t, const void *delta_t, const float *A,
                             const void *B_t, const void *C_t, const float *skip, const void *z_t,
                             void *y_t, int64_t batch, int64_t D, int64_t N, int64_t ld_xd,
                             int64_t ld_bc, int64_t ld_z, int64_t ld_y, jscan_a_form a_form,
                             jscan_dtype dtype, void *stream);

/*
 * Root-mean-square norm with the residual's addition in front of it, row by row (token by token):
 *     total = x + residual, rounded to `dtype` (the residual stream as it is kept)
 *     y = total gain / sqrt(mean_k total^2 + eps)
 * in fp32 (as (total gain) r with r = 1 / sqrt(...)), rounded once.  So the call on x and residual gives what the call on total
 * alone gives, bit for bit.  A row that holds a NaN or an infinity, or whose mean square plus eps is no normal fp32
 * number (the squares overflow, or eps is 0 and they vanish), has no norm: its y is NaN; no other row is touched.
 *   x, residual   M rows of K values in `dtype`, row strides ld_x, ld_residual >= K; residual may be NULL: total is then x
 *   gain          [K] fp32
 *   y             M rows out, stride ld_y
 *   total         M rows out, stride ld_total, or NULL when it is not wanted; goes with a residual.  It may be x or residual
 *                 itself (the same rows at the same stride)
 * 1 <= K <= 2^24, 0 <= M <= 2^30, eps >= 0; any K, any stride, pointers aligned to their elements.
 */
jscan_status jscan_rms_norm(const void *x, const void *residual, const float *gain, void *y,
                            void *total, int64_t M, int64_t K, int64_t ld_x, int64_t ld_residual,
                            int64_t ld_y, int64_t ld_total, float eps, jscan_dtype dtype, void *stream);

/*
 * The same with y in 8 bits, as jscan_quantize_rows would take it from y before it is rounded: the first input
 * of jscan_matmul_i8.  q [M][K] int8, 16-byte aligned; scale [M] fp32.  A row without a norm (see above) gets
 * scale NaN and q = 0.  K a multiple of 16, 16 <= K <= 131056.
 */
jscan_status jscan_rms_norm_quantize(const void *x, const void *residual, const float *gain, int8_t *q,
                                     float *scale, void *total, int64_t M, int64_t K, int64_t ld_x,
                                     int64_t ld_residual, int64_t ld_total, float eps,
                                     jscan_dtype dtype, void *stream);

/*
 * Backward pass of jscan_rms_norm from total.  With r = 1 / sqrt(mean total^2 + eps) and g = dy gain,
 *     dx = r (g - total r mean_k(g total r)) + dtotal,   dgain = sum over rows of dy total r
 * dx is the gradient of x and of residual alike.  Sums are fp32, in a fixed order (no atomics).  A row without a norm
 * (see above) has NaN for its dx and makes dgain NaN.
 *   dtotal      M rows, the gradient that comes from total's other uses, or NULL for zeros
 *   dx          M rows out; may be dtotal itself;   dgain [K] fp32 out (zeros with M == 0)
 *   workspace   jscan_rms_norm_backward_workspace(M, K) bytes, 16-byte aligned, overlapping nothing else.  Contents on
 *               entry do not matter.  Calls that share it must be ordered on one stream.
 */
jscan_status jscan_rms_norm_backward(const void *total, const float *gain, const void *dy,
                                     const void *dtotal, void *dx, float *dgain, int64_t M, int64_t K,
                                     int64_t ld_total, int64_t ld_dy, int64_t ld_dtotal, int64_t ld_dx,
                                     void *workspace, int64_t workspace_bytes, float eps,
                                     jscan_dtype dtype, void *stream);

/* Workspace bytes of jscan_rms_norm_backward for this shape (0 for a few short rows: it may then be NULL), or -1 if the
 * shape is invalid.  Host-only. */
int64_t jscan_rms_norm_backward_workspace(int64_t M, int64_t K);

/*
 * jscan_matmul_i8 with an epilogue: an activation of the scaled sum with its bias, then a residual,
 *     out[m][n] = act((sum_k q[m][k] w[n][k]) * q_scale[m] * w_scale[n] + bias[n]) + residual[m][n]
 * in fp32, rounded once.  activation is any jscan_activation (JSCAN_ERR_FORM otherwise).
 *   residual   M rows of N values in `dtype`, row stride ld_residual >= N, or NULL; it may be out itself (the same
 *              rows at the same stride)
 */
jscan_status jscan_matmul_i8_epilogue(const int8_t *q, const float *q_scale, const int8_t *w,
                                      const float *w_scale, const float *bias, const void *residual,
                                      void *out, int64_t M, int64_t N, int64_t K, int64_t ld_residual,
                                      int64_t ld_out, jscan_activation activation, jscan_dtype dtype,
                                      void *stream);

/* Static, human-readable name of a status code. */
const char *jscan_status_string(jscan_status s);

/* hipError_t behind the last JSCAN_ERR_HIP returned on the calling thread (0 if none). */
int jscan_last_hip_error(void);

/* Library ABI version: 100 * major + minor (101 adds the time-parallel prefill, 102 the
 * producer side, 103 the fused prefill, 104 the scaled-identity A entry points, 105 the
 * complex-valued state, 106 the exponential-trapezoidal rule, 107 the MIMO scan, 108 MIMO with the
 * trapezoidal rule, 109 the output row stride ld_y of the decode steps). */
int jscan_version(void);

#ifdef __cplusplus
}
#endif

#endif /* JSCAN_H */

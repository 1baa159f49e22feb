"""libjscan: the Mamba-1 (S6) selective state-space scan on AMD Instinct MI355X (gfx950).

The compute lives in hand-written HIP kernels behind the C ABI of ``include/jscan.h``;
this package only marshals torch tensors (device memory and streams) into those calls.
There is no CPU fallback: without the built library every call raises.

    y, h_final = prefill(x, delta, A, B, C)                # scan from the zero state
    y, h_final = prefill(x, delta, A, B, C, h0=h)          # resume from a state
    y_t = step(h, x_t, delta_t, A, B_t, C_t)               # one decode token, h in place
    y, h_final = prefill_chunked(x, delta, A, B, C)        # time-parallel, for few channels
    delta, B, C, d_low = ssm_inputs(x, w_x, g_d, g_B, g_C, w_dt, b_dt)   # producer side (MFMA)
    y, h_final = prefill_fused(x, d_low, w_dt, b_dt, A, B, C)             # delta computed in the scan
    y, h_final = prefill_scalar_a(x, delta, a, B, C)       # scaled-identity A (a: [D])
    y_t = step_scalar_a(h, x_t, delta_t, a, B_t, C_t)
    y, h_final = prefill_complex(x, delta, A, B, C)        # complex-valued state (pairs of states)
    y_t = step_complex(h, x_t, delta_t, A, B_t, C_t)
    y, h_final = prefill_trapezoid(x, delta, lam, A, B, C, form="diagonal")   # exponential-trapezoidal rule
    y_t = step_trapezoid(h, x_prev, B_prev, x_t, delta_t, lam_t, A, B_t, C_t)
    y, h_final = prefill_mimo(x, delta, A, B, C)          # R inputs and outputs per channel (MIMO)
    y_t = step_mimo(h, x_t, delta_t, A, B_t, C_t)
    y, h_final = prefill_mimo_trapezoid(x, delta, lam, A, B, C)   # both Mamba-3 changes together
    y_t = step_mimo_trapezoid(h, x_prev, B_prev, x_t, delta_t, lam_t, A, B_t, C_t)
    y, h_final = gated_scan(g, u, form="decay")            # gated recurrence: one state per channel
    dg, du, dh0 = gated_scan_backward(g, u, y, dy)         # its gradients
    states = gated_scan_states(g)                          # given to both: fp32 states behind bf16 gradients
    y_t = gated_step(h, g_t, u_t)                          # its decode token, h in place
    q, q_scale = quantize_rows(x)                          # activations to int8, a scale per token
    out = matmul_i8(q, q_scale, w, w_scale)                # int8 projection, a scale per output channel
    out = matmul_i8(q, q_scale, w, w_scale, activation="silu", residual=r)   # act(...) + r in its epilogue
    y, h_final = prefill_gate(x, delta, A, B, C, skip, z)  # (scan + skip x) silu(z) in one pass
    y_t = step_gate(h, x_t, delta_t, A, B_t, C_t, skip, z_t)
    y, total = rms_norm(x, gain, residual)                 # total = x + residual and its norm
    q, q_scale, total = rms_norm_quantize(x, gain, residual)   # the same into 8 bits, for matmul_i8
    dx, dgain = rms_norm_backward(total, gain, dy, dtotal) # its gradients
    y, state = causal_conv(x, w, bias, state)              # short causal convolution in front of a scan
    dx, dw, dbias, dstate = causal_conv_backward(x, w, dy, bias, state)   # its gradients
    y_t = causal_conv_step(state, x_t, w, bias)            # its decode token, the state in place
"""
from ._binding import (  # noqa: F401
    A_FORMS,
    ACTIVATIONS,
    D_STATE,
    GATE_FORMS,
    JScanError,
    causal_conv,
    causal_conv_backward,
    causal_conv_step,
    causal_conv_workspace_bytes,
    chunked_workspace_bytes,
    gated_scan,
    gated_scan_backward,
    gated_scan_states,
    gated_scan_workspace_bytes,
    gated_step,
    library,
    library_path,
    matmul_i8,
    prefill,
    prefill_chunked,
    prefill_chunked_noalloc,
    prefill_complex,
    prefill_fused,
    prefill_gate,
    prefill_gate_workspace_bytes,
    prefill_mimo,
    prefill_mimo_trapezoid,
    prefill_scalar_a,
    prefill_trapezoid,
    quantize_rows,
    rms_norm,
    rms_norm_backward,
    rms_norm_quantize,
    rms_norm_workspace_bytes,
    ssm_inputs,
    step,
    step_complex,
    step_gate,
    step_mimo,
    step_mimo_trapezoid,
    step_raw,
    step_scalar_a,
    step_trapezoid,
)

"""Tensors that carry a tangent (forward-mode automatic differentiation) do not require gradients, and a call that does
not pass the tangent on would lose it without a word: it is refused, for every tensor of every call that refuses
tensors that require gradients.  CPU only: the check comes before the one for the device."""
import pytest
import torch
import torch.autograd.forward_ad as fa

import mamba_selective_scan_03_amd as jscan

X, V, W = torch.zeros(2, 4, 16), torch.zeros(16), torch.zeros(16, 4)
S, R, T = torch.zeros(2, 3, 16), torch.zeros(2, 16), torch.zeros(2)
A, B, H = torch.zeros(16, 16), torch.zeros(2, 4, 16), torch.zeros(2, 16, 16)
Q = torch.zeros(2, 16, dtype=torch.int8)

CALLS = {   # a call on a list of tensors (None: left out)
    "gated_scan": (lambda g, u, h0: jscan.gated_scan(g, u, h0=h0), [X, X, R]),
    "gated_scan_backward": (lambda g, u, y, dy, h0, dh: jscan.gated_scan_backward(g, u, y, dy, h0=h0, dh_final=dh), [X, X, X, X, R, R]),
    "gated_step": (lambda h, g, u: jscan.gated_step(h, g, u), [R, R, R]),
    "quantize_rows": (lambda x: jscan.quantize_rows(x), [X]),
    "matmul_i8": (lambda sq, sw, b, r: jscan.matmul_i8(Q, sq, Q, sw, bias=b, residual=r), [T, T, T, torch.zeros(2, 2)]),
    "prefill_gate": (lambda x, d, a, b, c, k, z, h: jscan.prefill_gate(x, d, a, b, c, skip=k, z=z, h0=h), [X, X, A, B, B, V, X, H]),
    "step_gate": (lambda h, x, d, a, b, c, k, z: jscan.step_gate(h, x, d, a, b, c, skip=k, z_t=z), [H, R, R, A, R, R, V, R]),
    "causal_conv": (lambda x, w, b, s: jscan.causal_conv(x, w, bias=b, state=s), [X, W, V, S]),
    "causal_conv_backward": (lambda x, w, dy, b, s, ds: jscan.causal_conv_backward(x, w, dy, bias=b, state=s, dstate_out=ds), [X, W, X, V, S, S]),
    "causal_conv_step": (lambda s, x, w, b: jscan.causal_conv_step(s, x, w, bias=b), [S, R, W, V]),
    "rms_norm": (lambda x, g, r: jscan.rms_norm(x, g, residual=r), [X, V, X]),
    "rms_norm_quantize": (lambda x, g, r: jscan.rms_norm_quantize(x, g, residual=r), [X, V, X]),
    "rms_norm_backward": (lambda t, g, dy, dt: jscan.rms_norm_backward(t, g, dy, dtotal=dt), [X, V, X, X]),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_with_a_tangent_is_refused(name):
    call, tensors = CALLS[name]
    with fa.dual_level():
        for i in range(len(tensors)):
            args = list(tensors)
            args[i] = fa.make_dual(args[i].clone(), torch.ones_like(args[i]))
            with pytest.raises(ValueError, match="forward-mode"):
                call(*args)
            with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):   # which does not switch it off
                call(*args)
            args[i] = args[i].detach()
            with pytest.raises(ValueError, match="CUDA"):
                call(*args)
        with pytest.raises(ValueError, match="CUDA"):   # tensors without one are not meant
            call(*tensors)
    with pytest.raises(ValueError, match="CUDA"):
        call(*tensors)


def test_a_function_of_the_users_own_may_call_them():
    class Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            jscan.causal_conv(x, W)

    with fa.dual_level(), pytest.raises(ValueError, match="CUDA"):
        Conv.apply(fa.make_dual(X.clone(), torch.ones_like(X)))

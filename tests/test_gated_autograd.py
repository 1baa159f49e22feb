"""The gated recurrence's and the int8 projection's calls are not recorded by autograd: tensors that require gradients
are refused where it records, not answered with a result that has lost them.  CPU only: the check comes
before the one for the device, which stops every other call here."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan

X = torch.zeros(2, 4, 16)
V = torch.zeros(2, 16)
Q = torch.zeros(2, 16, dtype=torch.int8)


def grad(t):
    return t.clone().requires_grad_()


CALLS = [
    lambda f: jscan.gated_scan(f(X), X), lambda f: jscan.gated_scan(X, f(X)), lambda f: jscan.gated_scan(X, X, h0=f(V)),
    lambda f: jscan.gated_scan_backward(f(X), X, X, X), lambda f: jscan.gated_scan_backward(X, X, X, f(X)),
    lambda f: jscan.gated_scan_backward(X, None, X, X, dh_final=f(V)),
    lambda f: jscan.gated_step(f(V), V, V), lambda f: jscan.gated_step(V, f(V), V), lambda f: jscan.gated_step(V, V, f(V)),
    lambda f: jscan.quantize_rows(f(X)), lambda f: jscan.matmul_i8(Q, f(V[:, 0]), Q, V[:, 0]),
    lambda f: jscan.matmul_i8(Q, V[:, 0], Q, f(V[:, 0])), lambda f: jscan.matmul_i8(Q, V[:, 0], Q, V[:, 0], bias=f(V[:, 0])),
]


@pytest.mark.parametrize("call", CALLS)
def test_refused_where_autograd_records(call):
    with pytest.raises(ValueError, match="autograd"):
        call(grad)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(grad)
    with pytest.raises(ValueError, match="CUDA"):
        call(lambda t: t)


def test_a_function_of_the_users_own_may_call_them():
    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, g, u):
            jscan.gated_scan(g, u)

    with pytest.raises(ValueError, match="CUDA"):
        Scan.apply(grad(X), grad(X))

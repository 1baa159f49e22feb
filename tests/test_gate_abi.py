"""Refusals of the gated scan's entry points (skip and output gate), before any launch (the addresses below are never
dereferenced), and of their binding.  CPU only."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EALIAS, EHIP, EWORKSPACE, EFORM = range(9)
F32, BF16 = 0, 1
P = 0x100000000
S = 0x10000000


def prefill(**kw):
    a = dict(x=P, delta=P + S, A=P + 2 * S, B=P + 3 * S, C=P + 4 * S, h0=None, skip=P + 5 * S, z=P + 6 * S, y=P + 7 * S, h=P + 8 * S,
             batch=2, L=512, D=64, N=16, ld_z=64, chunk=-1, ws=None, ws_bytes=0, form=0, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_prefill_gate(*a.values(), None)


def step(**kw):
    a = dict(h=P, x=P + S, delta=P + 2 * S, A=P + 3 * S, B=P + 4 * S, C=P + 5 * S, skip=P + 6 * S, z=P + 7 * S, y=P + 8 * S, batch=2,
             D=64, N=16, ld_xd=64, ld_bc=16, ld_z=64, ld_y=64, form=0, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_step_gate(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(form=3), EFORM), (dict(dtype=2), EDTYPE), (dict(N=8), ESHAPE), (dict(D=60), ESHAPE), (dict(L=-1), ESHAPE),
    (dict(ld_z=56), ESHAPE), (dict(ld_z=65), ESHAPE), (dict(ld_z=(1 << 25) + 8), ESHAPE), (dict(chunk=-2), ESHAPE),
    (dict(skip=None, z=None), ENULL), (dict(x=None), ENULL), (dict(h=None), ENULL), (dict(y=None), ENULL),
    (dict(z=P + 6 * S + 8), EALIGN), (dict(skip=P + 5 * S + 2), EALIGN), (dict(x=P + 8), EALIGN),
    (dict(y=P + 6 * S), EALIAS), (dict(h=P + 6 * S), EALIAS), (dict(y=P + 5 * S), EALIAS), (dict(y=P), EALIAS), (dict(h=P + 5 * S), EALIAS),
    (dict(chunk=100, form=1), EFORM), (dict(chunk=100, form=2), EFORM), (dict(chunk=100), ENULL),
    (dict(chunk=100, ws=P + 9 * S, ws_bytes=10), EWORKSPACE), (dict(chunk=100, ws=P + 9 * S + 4, ws_bytes=1 << 40), EALIGN),
    (dict(chunk=100, ws=P + 6 * S, ws_bytes=1 << 40), EALIAS), (dict(chunk=100, ws=P + 5 * S, ws_bytes=1 << 40), EALIAS),
    (dict(batch=0), OK), (dict(D=0), OK),
])
def test_prefill_validation(kw, code):
    assert prefill(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(form=-1), EFORM), (dict(dtype=7), EDTYPE), (dict(N=4), ESHAPE), (dict(D=12), ESHAPE), (dict(ld_z=8), ESHAPE),
    (dict(ld_z=68), ESHAPE), (dict(ld_y=60), ESHAPE), (dict(ld_xd=70), ESHAPE), (dict(ld_bc=12), ESHAPE), (dict(h=None), ENULL),
    (dict(skip=None, z=None), ENULL), (dict(C=None), ENULL), (dict(z=P + 7 * S + 2), EALIGN), (dict(y=P + 8 * S + 8), EALIGN),
    (dict(y=P + 7 * S), EALIAS), (dict(z=P), EALIAS), (dict(skip=P + 64), EALIAS), (dict(y=P), EALIAS), (dict(y=P + 6 * S), EALIAS),
    (dict(batch=0), OK), (dict(D=0), OK),
])
def test_step_validation(kw, code):
    assert step(**kw) == code


def test_workspace_sizes():
    size = jscan.library().jscan_prefill_gate_workspace
    assert size(1, 100, 12, 16, 0) == -1 and size(1, 100, 64, 8, 0) == -1 and size(1, 100, 64, 16, -2) == -1 and size(-1, 9, 64, 16, 0) == -1
    assert size(1, 4096, 64, 16, -1) == 0 and size(0, 9, 64, 16, 0) == 0 and size(1, 1, 64, 16, 0) == 0
    assert size(1, 65536, 8192, 16, 0) == 0                     # enough channels to go token by token
    assert size(1, 4096, 64, 16, 256) == jscan.library().jscan_prefill_chunked_workspace(1, 4096, 64, 16, 256) > 0
    assert size(1, 65536, 1024, 16, 0) > 0 and size(1, 3932, 32, 16, 0) > 0
    # the limits: a plan that can be launched, or none
    for shape in ((1 << 20, 1000, 8), (1, (1 << 31) - 1, 8), (64, 1 << 20, 1 << 20), (1 << 20, 4096, 1 << 10)):
        assert size(*shape, 16, 0) >= 0


X, A, B, H = torch.zeros(2, 4, 8), torch.zeros(8, 16), torch.zeros(2, 4, 16), torch.zeros(2, 8, 16)
V = torch.zeros(8)


@pytest.mark.parametrize("call", [
    lambda f: jscan.prefill_gate(f(X), X, A, B, B, skip=V), lambda f: jscan.prefill_gate(X, X, A, B, B, skip=f(V)),
    lambda f: jscan.prefill_gate(X, X, A, B, B, z=f(X)), lambda f: jscan.prefill_gate(X, X, f(A), B, B, z=X),
    lambda f: jscan.step_gate(f(H), X[:, 0], X[:, 0], A, B[:, 0], B[:, 0], skip=V),
    lambda f: jscan.step_gate(H, X[:, 0], X[:, 0], A, B[:, 0], B[:, 0], z_t=f(X[:, 0])),
])
def test_refused_where_autograd_records(call):
    grad = lambda t: t.clone().requires_grad_()   # noqa: E731
    with pytest.raises(ValueError, match="autograd"):
        call(grad)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(grad)

"""Refusals of the norm's entry points and of the int8 product's epilogue, before any launch (the addresses below are
never dereferenced), and of their binding.  CPU only."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EALIAS, EHIP, EWORKSPACE, EFORM = range(9)
F32, BF16 = 0, 1
P = 0x100000000
S = 0x10000000


def norm(**kw):
    a = dict(x=P, res=P + S, gain=P + 2 * S, y=P + 3 * S, total=P + 4 * S, M=8, K=64, ld_x=64, ld_r=64, ld_y=64, ld_t=64, eps=1e-6,
             dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_rms_norm(*a.values(), None)


def quantize(**kw):
    a = dict(x=P, res=P + S, gain=P + 2 * S, q=P + 3 * S, scale=P + 5 * S, total=P + 4 * S, M=8, K=64, ld_x=64, ld_r=64, ld_t=64,
             eps=1e-6, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_rms_norm_quantize(*a.values(), None)


def backward(**kw):
    a = dict(total=P, gain=P + S, dy=P + 2 * S, dtotal=P + 3 * S, dx=P + 4 * S, dgain=P + 5 * S, M=16, K=64, ld_t=64, ld_dy=64, ld_dt=64,
             ld_dx=64, ws=P + 8 * S, ws_bytes=1 << 30, eps=1e-6, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_rms_norm_backward(*a.values(), None)


def product(**kw):
    a = dict(q=P, sq=P + S, w=P + 2 * S, sw=P + 3 * S, bias=None, res=P + 4 * S, out=P + 5 * S, M=8, N=64, K=64, ld_r=64, ld_o=64, act=1,
             dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_matmul_i8_epilogue(*a.values(), None)


COMMON = [
    (dict(dtype=2), EDTYPE), (dict(M=-1), ESHAPE), (dict(M=(1 << 30) + 1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=-16), ESHAPE),
    (dict(eps=-1.0), ESHAPE), (dict(eps=float("nan")), ESHAPE), (dict(ld_x=63), ESHAPE), (dict(ld_r=63), ESHAPE), (dict(ld_t=1), ESHAPE),
    (dict(x=None), ENULL), (dict(gain=None), ENULL), (dict(res=None), ENULL), (dict(x=P + 1), EALIGN), (dict(res=P + S + 1), EALIGN),
    (dict(gain=P + 2 * S + 2), EALIGN), (dict(total=P + 4 * S + 1), EALIGN), (dict(total=P + 64), EALIAS),
    (dict(total=P, ld_t=128, ld_x=130), EALIAS), (dict(total=P + 2 * S), EALIAS), (dict(M=0, x=None, gain=None), OK),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(ld_y=60), ESHAPE), (dict(y=None), ENULL), (dict(y=P + 3 * S + 1), EALIGN), (dict(y=P), EALIAS), (dict(y=P + S), EALIAS),
    (dict(y=P + 4 * S), EALIAS), (dict(y=P + 2 * S), EALIAS), (dict(K=(1 << 24) + 1, ld_x=1 << 25, ld_r=1 << 25, ld_y=1 << 25, ld_t=1 << 25), ESHAPE)])
def test_norm_validation(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(K=40), ESHAPE), (dict(K=131072, ld_x=131072, ld_r=131072, ld_t=131072), ESHAPE), (dict(q=None), ENULL), (dict(scale=None), ENULL),
    (dict(q=P + 3 * S + 8), EALIGN), (dict(scale=P + 5 * S + 2), EALIGN), (dict(q=P), EALIAS), (dict(scale=P + S), EALIAS),
    (dict(scale=P + 3 * S), EALIAS), (dict(q=P + 4 * S), EALIAS)])
def test_quantize_validation(kw, code):
    assert quantize(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), EDTYPE), (dict(M=-1), ESHAPE), (dict(K=0), ESHAPE), (dict(ld_t=60), ESHAPE), (dict(ld_dy=60), ESHAPE),
    (dict(ld_dt=60), ESHAPE), (dict(ld_dx=60), ESHAPE), (dict(eps=-1e-3), ESHAPE), (dict(total=None), ENULL), (dict(dy=None), ENULL),
    (dict(dx=None), ENULL), (dict(gain=None), ENULL), (dict(dgain=None), ENULL), (dict(M=0, dgain=None), ENULL),
    (dict(ws=None), EWORKSPACE), (dict(ws_bytes=4), EWORKSPACE), (dict(ws=P + 8 * S + 4), EALIGN), (dict(dgain=P + 5 * S + 1), EALIGN),
    (dict(dx=P + 1), EALIGN), (dict(dx=P), EALIAS), (dict(dx=P + 2 * S), EALIAS), (dict(dx=P + 3 * S + 2), EALIAS),
    (dict(dx=P + 3 * S, ld_dx=65), EALIAS), (dict(dgain=P + S), EALIAS), (dict(ws=P), EALIAS), (dict(ws=P + 5 * S), EALIAS)])
def test_backward_validation(kw, code):
    assert backward(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(act=3), EFORM), (dict(act=-1), EFORM), (dict(dtype=5), EDTYPE), (dict(K=24), ESHAPE), (dict(ld_r=63), ESHAPE),
    (dict(ld_o=63), ESHAPE), (dict(q=None), ENULL), (dict(out=None), ENULL), (dict(res=P + 4 * S + 1), EALIGN), (dict(res=P + 5 * S + 2), EALIAS),
    (dict(res=P + 5 * S, ld_r=66), EALIAS), (dict(out=P), EALIAS), (dict(M=0), OK), (dict(N=0), OK)])
def test_product_validation(kw, code):
    assert product(**kw) == code


def test_workspace_sizes():
    size = jscan.library().jscan_rms_norm_backward_workspace
    assert size(-1, 64) == -1 and size(8, 0) == -1 and size(0, 64) == 0 and size(3, 64) == 0 and 0 < size(16, 64) <= 16 * 64 * 4
    assert size(16384, 4096) <= 0.1 * 4 * 16384 * 4096 * 2


X, V = torch.zeros(2, 4, 16), torch.zeros(16)
Q = torch.zeros(2, 16, dtype=torch.int8)


@pytest.mark.parametrize("call", [
    lambda f: jscan.rms_norm(f(X), V), lambda f: jscan.rms_norm(X, f(V)), lambda f: jscan.rms_norm(X, V, residual=f(X)),
    lambda f: jscan.rms_norm_quantize(f(X), V), lambda f: jscan.rms_norm_backward(X, V, f(X)),
    lambda f: jscan.rms_norm_backward(X, V, X, dtotal=f(X)), lambda f: jscan.matmul_i8(Q, V[:2], Q, V[:2], residual=f(V[:4].view(2, 2))),
])
def test_refused_where_autograd_records(call):
    grad = lambda t: t.clone().requires_grad_()   # noqa: E731
    with pytest.raises(ValueError, match="autograd"):
        call(grad)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(grad)


def test_binding_refuses_an_unknown_activation():
    with pytest.raises(ValueError, match="activation"):
        jscan.matmul_i8(Q, V[:2], Q, V[:2], activation="relu")

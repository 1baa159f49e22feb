"""Refusals of the short causal convolution's entry points, before any launch (the addresses below are never
dereferenced), and of their binding.  CPU only."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EALIAS, EHIP, EWORKSPACE, EFORM = range(9)
F32, BF16 = 0, 1
P = 0x100000000
S = 0x10000000


def conv(**kw):
    a = dict(x=P, state=None, w=P + S, bias=None, n=None, y=P + 2 * S, out=None, batch=2, L=64, D=64, W=4, ld_x=64, ld_y=64,
             act=1, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_causal_conv(*a.values(), None)


def backward(**kw):
    a = dict(x=P, state=None, w=P + S, bias=None, n=None, dy=P + 2 * S, dso=None, dx=P + 3 * S, ds=None, dw=P + 4 * S, db=None,
             batch=2, L=64, D=64, W=4, ld_x=64, ld_dy=64, ld_dx=64, ws=P + 8 * S, ws_bytes=1 << 40, act=1, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_causal_conv_backward(*a.values(), None)


def step(**kw):
    a = dict(state=P, x=P + S, w=P + 2 * S, bias=None, y=P + 3 * S, batch=2, D=64, W=4, ld_x=64, ld_y=64, act=1, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_causal_conv_step(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(act=2), EFORM), (dict(act=-1), EFORM), (dict(dtype=3), EDTYPE), (dict(W=1), ESHAPE), (dict(W=5), ESHAPE),
    (dict(batch=-1), ESHAPE), (dict(L=-1), ESHAPE), (dict(D=-1), ESHAPE), (dict(D=(1 << 24) + 1), ESHAPE), (dict(L=1 << 31), ESHAPE),
    (dict(batch=(1 << 20) + 1), ESHAPE), (dict(ld_x=63), ESHAPE), (dict(ld_y=0), ESHAPE), (dict(ld_x=1 << 58), ESHAPE),
    (dict(x=None), ENULL), (dict(y=None), ENULL), (dict(w=None), ENULL), (dict(x=P + 1), EALIGN),
    (dict(dtype=F32, y=P + 2 * S + 2), EALIGN), (dict(w=P + S + 2), EALIGN), (dict(bias=P + 5 * S + 1), EALIGN),
    (dict(n=P + 5 * S + 2), EALIGN), (dict(state=P + 5 * S + 1), EALIGN), (dict(out=P + 5 * S + 1), EALIGN),
    (dict(y=P), EALIAS), (dict(y=P + 128), EALIAS), (dict(y=P + S), EALIAS), (dict(out=P + 2 * S), EALIAS), (dict(out=P), EALIAS),
    (dict(state=P + 5 * S, out=P + 5 * S + 2), EALIAS), (dict(y=P + 5 * S, n=P + 5 * S), EALIAS),
    (dict(y=P + 130, ld_x=128, ld_y=130), EALIAS), (dict(batch=0, x=None, y=None, w=None), OK), (dict(D=0, w=None), OK),
])
def test_conv_validation(kw, code):
    assert conv(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(act=2), EFORM), (dict(dtype=2), EDTYPE), (dict(W=0), ESHAPE), (dict(ld_dy=1), ESHAPE), (dict(ld_dx=60), ESHAPE),
    (dict(x=None), ENULL), (dict(dy=None), ENULL), (dict(dx=None), ENULL), (dict(dw=None), ENULL), (dict(w=None), ENULL),
    (dict(ws=None), EWORKSPACE), (dict(ws_bytes=100), EWORKSPACE), (dict(ws=P + 8 * S + 8), EALIGN), (dict(dw=P + 4 * S + 2), EALIGN),
    (dict(dx=P + 3 * S + 1), EALIGN), (dict(dx=P), EALIAS), (dict(dx=P + 2 * S), EALIAS), (dict(dw=P + S), EALIAS),
    (dict(ws=P), EALIAS), (dict(db=P + 4 * S), EALIAS), (dict(dso=P + 5 * S, ds=P + 5 * S), EALIAS),
    (dict(ws=P + 3 * S), EALIAS), (dict(D=0), OK),
])
def test_backward_validation(kw, code):
    assert backward(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(act=3), EFORM), (dict(dtype=9), EDTYPE), (dict(W=6), ESHAPE), (dict(ld_x=3), ESHAPE), (dict(ld_y=3), ESHAPE),
    (dict(state=None), ENULL), (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL), (dict(state=P + 1), EALIGN),
    (dict(y=P + S), EALIAS), (dict(y=P), EALIAS), (dict(x=P + 64), EALIAS), (dict(w=P + 4), EALIAS), (dict(batch=0, state=None), OK),
    (dict(D=0), OK),
])
def test_step_validation(kw, code):
    assert step(**kw) == code


def test_workspace_sizes():
    size = jscan.library().jscan_causal_conv_backward_workspace
    assert size(2, 64, 64, 5) == -1 and size(-1, 64, 64, 4) == -1 and size(0, 64, 64, 4) == 0 and size(2, 64, 0, 4) == 0
    assert size(1, 1, 8, 4) == 5 * 8 * 4   # one share of every tap and the bias
    # few percent of the tensors it stands beside
    assert size(8, 4096, 8192, 4) < 0.05 * 3 * 8 * 4096 * 8192 * 2
    # no overflow at the limits
    assert size(1 << 20, (1 << 31) - 1, 64, 4) > 0 and size(1, (1 << 31) - 1, 1 << 24, 4) > 0


X, V = torch.zeros(2, 5, 6), torch.zeros(6, 4)


@pytest.mark.parametrize("call", [
    lambda f: jscan.causal_conv(f(X), V), lambda f: jscan.causal_conv(X, f(V)), lambda f: jscan.causal_conv(X, V, bias=f(X[0, 0])),
    lambda f: jscan.causal_conv(X, V, state=f(X[:, :3])), lambda f: jscan.causal_conv_backward(X, V, f(X)),
    lambda f: jscan.causal_conv_backward(X, f(V), X), lambda f: jscan.causal_conv_step(f(X[:, :3].contiguous()), X[:, 0], V),
    lambda f: jscan.causal_conv_step(X[:, :3].contiguous(), X[:, 0], f(V)),
])
def test_refused_where_autograd_records(call):
    grad = lambda t: t.clone().requires_grad_()   # noqa: E731
    with pytest.raises(ValueError, match="autograd"):
        call(grad)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(grad)


def test_binding_refuses_other_activations():
    for call in (lambda a: jscan.causal_conv(X, V, activation=a), lambda a: jscan.causal_conv_backward(X, V, X, activation=a),
                 lambda a: jscan.causal_conv_step(X[:, :3], X[:, 0], V, activation=a)):
        for a in ("gelu_tanh", "relu", None):
            with pytest.raises(ValueError, match="activation"):
                call(a)

"""Saved states of the gated recurrence: refusals before any launch (the addresses below are never dereferenced) and
what the rounding of y does to the gradients.  CPU only."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from oracle import gated as O

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EALIAS, EHIP, EWORKSPACE, EFORM = range(9)
F32, BF16 = 0, 1
P = 0x100000000
STEP = 0x10000000


def save(**kw):
    a = dict(g=P, u=P + STEP, h0=None, n=None, y=P + 2 * STEP, h=P + 3 * STEP, states=P + 4 * STEP, batch=2, L=64, D=64,
             ld_g=64, ld_u=64, ld_y=64, ws=P + 8 * STEP, ws_bytes=1 << 40, form=0, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_gated_scan_save(*a.values(), None)


def backward(**kw):
    a = dict(g=P, u=P + STEP, states=P + 2 * STEP, dy=P + 3 * STEP, dh=None, n=None, dg=P + 4 * STEP, du=P + 5 * STEP,
             dh0=None, batch=2, L=64, D=64, ld_g=64, ld_u=64, ld_dy=64, ld_dg=64, ld_du=64, ws=P + 8 * STEP,
             ws_bytes=1 << 40, form=0, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_gated_scan_backward_saved(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(form=2), EFORM), (dict(dtype=F32), EDTYPE), (dict(dtype=7), EDTYPE), (dict(L=-1), ESHAPE), (dict(ld_y=63), ESHAPE),
    (dict(states=None), ENULL), (dict(h=None), ENULL), (dict(states=P + 4 * STEP + 8), EALIGN), (dict(states=P + STEP), EALIAS),
    (dict(states=P + 2 * STEP + 64), EALIAS), (dict(h=P + 4 * STEP + 2 * 8 * 64 * 4 - 4), EALIAS), (dict(h0=P + 4 * STEP), EALIAS),
    (dict(batch=0, states=None), OK), (dict(D=0), OK),
])
def test_scan_validation(kw, code):
    assert save(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(form=9), EFORM), (dict(dtype=F32), EDTYPE), (dict(D=-1), ESHAPE), (dict(ld_u=60), ESHAPE), (dict(ld_du=1), ESHAPE),
    (dict(states=None), ENULL), (dict(u=None), ENULL), (dict(dy=None), ENULL), (dict(dg=None), ENULL),
    (dict(states=P + 2 * STEP + 4), EALIGN), (dict(du=P + 5 * STEP + 1), EALIGN), (dict(dg=P + 2 * STEP), EALIAS),
    (dict(dh0=P + 2 * STEP + 128), EALIAS), (dict(du=P + STEP), EALIAS), (dict(dh=P + 6 * STEP, dh0=P + 6 * STEP + 256), EALIAS),
    (dict(batch=0, states=None), OK), (dict(D=0), OK),
])
def test_backward_validation(kw, code):
    assert backward(**kw) == code


def test_sizes():
    size = jscan.library().jscan_gated_scan_states
    assert size(2, 64, 64) == 2 * 8 * 64 * 4 and size(3, 65, 7) == 3 * 9 * 7 * 4 and size(0, 9, 9) == 0 and size(4, 0, 8) == 0
    assert size(-1, 8, 8) == -1 and size(1, 1 << 31, 8) == -1 and size(1 << 12, (1 << 31) - 1, 1 << 24) == -1
    g = torch.zeros(2, 9, 5, dtype=torch.bfloat16)
    assert jscan.gated_scan_states(g).shape == (2, 2, 5) and jscan.gated_scan_states(g).dtype == torch.float32
    assert jscan.gated_scan_states(g.float()) is None
    with pytest.raises(ValueError):
        jscan.gated_scan_states(g.half())


@pytest.mark.parametrize("form", ["decay", "sigmoid"])
def test_what_rounding_y_does_to_the_gradient_of_the_gate(form):
    """dg from y rounded to bf16 is off by at most 2^-8 of |c h| (sigmoid: of |c (1 - a) h|), and for inputs close to the
    state that is no small part of the sigmoid form's dg, which is why states can be kept."""
    r = np.random.default_rng(1)
    L, D = 256, 16
    g = -np.exp(r.normal(-1, 1, (1, L, D))) if form == "decay" else 2 + 1.5 * r.standard_normal((1, L, D))
    u, dy = 3 + 0.1 * r.standard_normal((1, L, D)), r.standard_normal((1, L, D))
    h0 = np.full((1, D), 3.0)
    y, _ = O.scan(g, u, h0, None, form)
    rounded = torch.from_numpy(y).to(torch.bfloat16).double().numpy()
    dg, _, _, c = O.backward(g, u, y, dy, h0, None, None, form)
    off = np.abs(O.backward(g, u, rounded, dy, h0, None, None, form)[0] - dg)
    before = np.concatenate([h0[:, None], y[:, :-1]], 1)
    assert (off <= 2.0 ** -8 * np.abs(c * O.gates(g, form)[1] * before) * (1 + 1e-9)).all()
    relative = off > 2.0 ** -7 * np.abs(dg)
    assert relative.mean() > 0.5 if form == "sigmoid" else not relative.any()

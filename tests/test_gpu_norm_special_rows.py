"""Rows that have no root-mean-square norm, on the GPU: a NaN or an infinity among them, or a mean square plus eps that is
no normal fp32 number (the squares overflow, or eps is 0 and they vanish).  They are NaN in every form of the call, and
no other row is touched.  Rows next to those borders keep the oracle's bounds."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits, f64
from oracle import layer as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NONE = {1: 1e30, 3: 0.0, 5: 1e-25, 7: 1e-19, 9: float("inf")}   # row: its values (eps 0)
SMALL, LARGE = 4e-19, 5e16   # mean squares of 1.6e-37 and, over 65536 values, a sum of 1.6e38


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def rows(K, dtype, seed=0):
    x = normal(seed, 12, K)
    for m, v in NONE.items():
        x[m] = v
    x[9, 1:] = 1.0   # one infinity
    x[2], x[4] = SMALL, LARGE
    return x.to(DT[dtype]).cuda()


# a piece and less, one, four and sixteen waves, rows read again, rows element by element
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [3, 48, 1008, 4096, 10000, 20000, 65536])
def test_rows_without_a_norm_are_nan_and_alone(K, dtype):
    x, gain = rows(K, dtype), (1 + 0.3 * normal(3, K)).cuda()
    good = [m for m in range(12) if m not in NONE]
    y, _ = jscan.rms_norm(x, gain, eps=0.0)
    assert torch.isnan(y[list(NONE)]).all()
    want, err = O.rms_norm(x[good], gain, 0.0)
    tol = err + torch.finfo(y.dtype).eps / 2 * (np.abs(want) + err)
    assert (np.abs(f64(y[good]) - want) <= tol).all()
    alone, _ = jscan.rms_norm(x[good], gain, eps=0.0)
    assert torch.equal(bits(y[good]), bits(alone))
    if K % 16 == 0:
        q, s, _ = jscan.rms_norm_quantize(x, gain, eps=0.0)
        assert torch.isnan(s[list(NONE)]).all() and not q[list(NONE)].any() and torch.isfinite(s[good]).all()
        q0, s0, _ = jscan.rms_norm_quantize(x[good], gain, eps=0.0)
        assert torch.equal(q[good], q0) and torch.equal(bits(s[good]), bits(s0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [3, 48, 1008, 4096, 10000, 20000, 65536])
def test_their_gradients_are_nan_and_alone(K, dtype):
    x, gain, dy = rows(K, dtype, 1), (1 + 0.3 * normal(3, K)).cuda(), normal(4, 12, K).to(DT[dtype]).cuda()
    good = [m for m in range(12) if m not in NONE]
    dx, dgain = jscan.rms_norm_backward(x, gain, dy, dtotal=dy, eps=0.0)
    assert torch.isnan(dx[list(NONE)]).all() and torch.isnan(dgain).all()
    alone, sums = jscan.rms_norm_backward(x[good], gain, dy[good], dtotal=dy[good], eps=0.0)
    assert torch.equal(bits(dx[good]), bits(alone)) and torch.isfinite(sums).all()


def test_a_vanishing_row_has_a_norm_where_eps_is_normal():
    x, gain = torch.zeros(2, 64, device="cuda"), torch.ones(64, device="cuda")
    for eps in (1e-6, 2.0 ** -126):
        y, _ = jscan.rms_norm(x, gain, eps=eps)
        dx, dgain = jscan.rms_norm_backward(x, gain, x + 1, eps=eps)
        assert not y.any() and not dgain.any() and torch.isfinite(dx).all()

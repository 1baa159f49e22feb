"""Infinities and NaN in the gated recurrence stay where the recurrence carries them: in their channel and their
sequence, forward from an input or a starting state, backward from dy, past a reset too.  Every other value
has the bits of the run without them, in each layout of the scan (one wave, several, narrow strips, cut)."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits
from test_gpu_gated_scan import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["decay", "sigmoid"])
@pytest.mark.parametrize("dtype,L,D", [("bf16", 8, 66), ("f32", 30, 40), ("bf16", 300, 66), ("f32", 600, 34), ("bf16", 9000, 64),
                                       ("bf16", 4097, 2047), ("f32", 3000, 1024)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_stay_in_their_channel_and_sequence(dtype, L, D, value, form):
    g, u, dy, h0, dh = make(3, L, D, dtype, form, L + D)
    reset, at, c = 5 * L // 8, L // 4, D // 2 + 1
    g[:, reset] = -float("inf")

    def run(u, dy, h0, states):
        y, h = jscan.gated_scan(g, u, h0=h0, form=form, states=states)
        return (y, h, *jscan.gated_scan_backward(g, u, y, dy, h0=h0, dh_final=dh, form=form, states=states))

    for states in (None, jscan.gated_scan_states(g)):
        want = run(u, dy, h0, states)
        u2, dy2, h02 = u.clone(), dy.clone(), h0.clone()
        u2[1, at, c], dy2[1, L - 1 - at, c - 1], h02[2, 0] = value, value, value
        y, h, dg, du, dh0 = run(u2, dy2, h02, states)
        # from the input on, past the reset (0 times an infinity is NaN); from dy back; from the starting state on
        assert not torch.isfinite(y[1, at, c]) and torch.isnan(y[1, reset:, c]).all() and torch.isnan(h[1, c])
        assert torch.isnan(y[2, reset:, 0]).all() and torch.isnan(h[2, 0])
        assert torch.isnan(du[1, :min(reset, L - 1 - at), c - 1]).all() and torch.isnan(dh0[1, c - 1])
        same = torch.ones(3, L, D, dtype=torch.bool)
        same[1, :, c - 1:c + 1] = same[2, :, 0] = False
        state = torch.ones(3, D, dtype=torch.bool)
        state[1, c - 1:c + 1] = state[2, 0] = False
        for a, b, keep in zip((y, h, dg, du, dh0), want, (same, state, same, same, state)):
            assert torch.equal(bits(a)[keep], bits(b)[keep])
        assert torch.equal(bits(y)[1, :at, c], bits(want[0])[1, :at, c])

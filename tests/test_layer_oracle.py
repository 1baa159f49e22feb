"""The fp64 oracle of the layer's operators against closed forms and differences.  CPU only."""
import numpy as np
import pytest

from oracle import layer as O


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_a_pulse_walks_through_the_taps(W):
    w = rng(W).standard_normal((3, W))
    x = np.zeros((1, 8, 3))
    x[0, 2] = 1
    y, out, _ = O.conv(x, w, act="none")
    want = np.zeros((8, 3))
    want[2:2 + W] = w[:, ::-1].T   # the token itself by the last tap, the next by the one before
    assert np.array_equal(y[0], want) and not out.any()


def test_state_and_tokens_are_one_sequence():
    r = rng(1)
    x, w, b = r.standard_normal((2, 9, 5)), r.standard_normal((5, 4)), r.standard_normal(5)
    y, out, _ = O.conv(x, w, b)
    for cut in (1, 2, 3, 8):
        y0, mid, _ = O.conv(x[:, :cut], w, b)
        y1, end, _ = O.conv(x[:, cut:], w, b, state=mid)
        assert np.allclose(np.concatenate([y0, y1], 1), y, rtol=1e-14) and np.array_equal(end, out)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradients_against_differences(act):
    r = rng(2)
    x, w, b, s = (r.standard_normal(v) for v in ((2, 6, 3), (3, 4), (3,), (2, 3, 3)))
    dy, ds, n = r.standard_normal((2, 6, 3)), r.standard_normal((2, 3, 3)), np.array([6, 2])

    def loss(x, w, b, s):
        y, out, _ = O.conv(x, w, b, s, n, act)
        return (y * dy).sum() + (out * ds).sum()

    g, _ = O.conv_backward(x, w, dy, b, s, ds, n, act)
    for k, (i, name) in enumerate([(0, "dx"), (1, "dw"), (2, "dbias"), (3, "dstate")]):
        args = [x, w, b, s]
        for _ in range(12):
            step = r.standard_normal(args[i].shape)
            hi, lo = list(args), list(args)
            hi[i], lo[i] = args[i] + 1e-5 * step, args[i] - 1e-5 * step
            want = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(want - (g[name] * step).sum()) < 1e-8 * (1 + np.abs(g[name] * step).sum())

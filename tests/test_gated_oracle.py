"""Pins of the gated recurrence's and the int8 projection's oracle: values fixed by arithmetic, by
finite differences or by structure, not by re-running its formulas.  CPU only."""
import numpy as np
import pytest

from oracle import gated as O


def _inputs(batch, L, D, form, seed):
    r = np.random.default_rng(seed)
    g = -np.exp(r.normal(-1, 1, (batch, L, D))) if form == "decay" else r.normal(1, 2, (batch, L, D))
    return g, r.standard_normal((batch, L, D)), r.standard_normal((batch, D))


def test_zero_log_gate_is_a_running_sum():
    u = np.arange(1.0, 13.0).reshape(1, 4, 3)
    y, h = O.scan(np.zeros((1, 4, 3)), u, h0=np.full((1, 3), 10.0))
    assert np.array_equal(y, 10 + np.cumsum(u, 1)) and np.array_equal(h, y[:, -1])


def test_constant_gate_is_a_geometric_series():
    L, a = 9, 0.75
    y, _ = O.scan(np.full((1, L, 1), np.log(a)), np.ones((1, L, 1)))
    want = (1 - a ** np.arange(1, L + 1)) / (1 - a)
    assert np.allclose(y[0, :, 0], want, rtol=1e-14)
    y, _ = O.scan(np.full((1, L, 1), np.log(a / (1 - a))), np.ones((1, L, 1)), form="sigmoid")
    assert np.allclose(y[0, :, 0], 1 - a ** np.arange(1, L + 1), rtol=1e-14)


@pytest.mark.parametrize("form", ["decay", "sigmoid"])
def test_minus_infinity_resets_and_lengths_stop(form):
    g, u, h0 = _inputs(2, 8, 3, form, 1)
    g[:, 5] = -np.inf
    y, h = O.scan(g, u, h0, form=form)
    tail, h2 = O.scan(g[:, 5:], u[:, 5:], None, form=form)
    assert np.array_equal(y[:, 5:], tail) and np.array_equal(h, h2)
    y3, h3 = O.scan(g, u, h0, lengths=np.array([4, 0]), form=form)
    assert np.array_equal(y3[0, :4], y[0, :4]) and not y3[0, 4:].any() and not y3[1].any()
    assert np.array_equal(h3[0], y[0, 3]) and np.array_equal(h3[1], h0[1])


@pytest.mark.parametrize("form", ["decay", "sigmoid"])
@pytest.mark.parametrize("lengths", [None, [7, 0, 3]])
def test_gradients_match_central_differences(form, lengths):
    batch, L, D = 3, 7, 2
    g, u, h0 = _inputs(batch, L, D, form, 2)
    r = np.random.default_rng(3)
    wy, wh = r.standard_normal((batch, L, D)), r.standard_normal((batch, D))
    n = None if lengths is None else np.array(lengths)

    def loss(g, u, h0):
        y, h = O.scan(g, u, h0, n, form)
        return np.sum(wy * y) + np.sum(wh * h)

    y, _ = O.scan(g, u, h0, n, form)
    dg, du, dh0, _ = O.backward(g, u, y, wy, h0, wh, n, form)
    eps = 1e-6
    for got, k in ((dg, 0), (du, 1), (dh0, 2)):
        args = [g, u, h0]
        for i in np.ndindex(args[k].shape):
            up, dn = [v.copy() for v in args], [v.copy() for v in args]
            up[k][i] += eps
            dn[k][i] -= eps
            assert got[i] == pytest.approx((loss(*up) - loss(*dn)) / (2 * eps), rel=1e-7, abs=1e-8)


@pytest.mark.parametrize("form", ["decay", "sigmoid"])
def test_error_bounds_hold_for_fp32_scans_and_are_not_slack(form):
    """The running error bounds against the same recurrence evaluated in fp32 numpy, in two orders
    (token by token, and by halves): within the bound, and the bound within 1e-4 of the values."""
    g, u, h0 = _inputs(2, 300, 16, form, 4)
    g, u, h0 = (v.astype(np.float32) for v in (g, u, h0))
    y, _ = O.scan(g, u, h0, form=form)
    E, M = O.scan_error(g, u, h0, form=form)
    f = np.float32
    a = np.exp(g) if form == "decay" else f(1) / (f(1) + np.exp(-g))
    x = u if form == "decay" else u / (f(1) + np.exp(g))
    h, seq = h0.copy(), np.zeros_like(u)
    for t in range(u.shape[1]):
        h = a[:, t] * h + x[:, t]
        seq[:, t] = h

    def halves(a, x):
        if a.shape[1] == 1:
            return a, x
        k = a.shape[1] // 2
        (a1, x1), (a2, x2) = halves(a[:, :k], x[:, :k]), halves(a[:, k:], x[:, k:])
        return np.concatenate([a1, a2 * a1[:, -1:]], 1), np.concatenate([x1, x2 + a2 * x1[:, -1:]], 1)

    A, X = halves(a, x)
    for got in (seq, X + A * h0[:, None]):
        assert (np.abs(got - y) <= E).all()
    assert (E <= 1e-4 * M + 1e-6).all()


def test_quantiser_hand_values():
    x = np.zeros((4, 16))
    x[0, :4] = [127, -127, 0.5, 1.5]        # scale 1: ties go to even
    x[1, 0] = 1e-45                         # far below the smallest scale
    x[2, 3] = np.nan
    q, s = O.quantize_rows(x)
    assert list(q[0, :4]) == [127, -127, 0, 2] and s[0] == 1
    assert not q[1].any() and s[1] == np.float32(2.0 ** -126)
    assert not q[2].any() and np.isnan(s[2])
    assert not q[3].any() and s[3] == np.float32(2.0 ** -126)


def test_product_hand_values():
    q = np.array([[1, -2] + [0] * 14, [127] * 16], np.int8)
    w = np.array([[3, 4] + [0] * 14, [-128] * 16], np.int8)
    out = O.matmul_i8(q, np.array([0.5, 1.0]), w, np.array([2.0, 1.0]), np.array([0.0, 1.0]))
    assert np.array_equal(out, [[-5.0, 0.5 * 128 + 1], [2.0 * 889, -127 * 128 * 16 + 1]])

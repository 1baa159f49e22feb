"""fp64 oracle of the gated recurrence, its gradients and its forward error bounds, and of the int8
projection (numpy, token by token; shares no code with the GPU path).

    decay    a = exp(g),      b = 1        h_t = a_t h_{t-1} + b_t u_t
    sigmoid  a = sigmoid(g),  b = 1 - a    y_t = h_t
"""
from __future__ import annotations

import numpy as np


def _f64(t):
    return np.asarray(t.detach().double().cpu().numpy() if hasattr(t, "detach") else t, np.float64)


def gates(g, form):
    g = _f64(g)
    if form == "decay":
        return np.exp(g), np.ones_like(g)
    with np.errstate(over="ignore"):   # exp(inf) = inf: the far end of the sigmoid is an exact 0
        return 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))


def _lengths(lengths, batch, L):
    return np.full(batch, L) if lengths is None else np.clip(np.asarray(_f64(lengths), np.int64), 0, L)


def scan(g, u, h0=None, lengths=None, form="decay"):
    """(y [batch, L, D], h_final [batch, D]); y is zero in the padding."""
    a, b = gates(g, form)
    u = _f64(u)
    batch, L, D = u.shape
    n = _lengths(lengths, batch, L)
    h = np.zeros((batch, D)) if h0 is None else _f64(h0).copy()
    y = np.zeros_like(u)
    for t in range(L):
        on = t < n
        h[on] = a[on, t] * h[on] + b[on, t] * u[on, t]
        y[on, t] = h[on]
    return y, h


def backward(g, u, y, dy, h0=None, dh_final=None, lengths=None, form="decay"):
    """(dg, du, dh0, c) with h_{t-1} taken from y; c_t = a_t dL/dh_t."""
    a, b = gates(g, form)
    y, dy, u = _f64(y), _f64(dy), None if u is None else _f64(u)
    batch, L, D = y.shape
    n = _lengths(lengths, batch, L)
    c = np.zeros((batch, D)) if dh_final is None else _f64(dh_final).copy()
    start = np.zeros((batch, D)) if h0 is None else _f64(h0)
    dg, du, cs = np.zeros_like(y), np.zeros_like(y), np.zeros_like(y)
    for t in reversed(range(L)):
        on = t < n
        before = (y[:, t - 1] if t else start)[on]
        G = dy[on, t] + c[on]
        c[on] = a[on, t] * G
        cs[on, t] = c[on]
        du[on, t] = b[on, t] * G
        dg[on, t] = c[on] * before if form == "decay" else c[on] * b[on, t] * (before - u[on, t])
    return dg, du, c, cs


def gate_error(g):
    """Relative error of a gate evaluated in fp32 as the kernels do: an exponential accurate to one
    unit (2^-23) of an argument rounded once (|g| log2(e) 2^-24 in the exponent, so |g| 2^-24
    relative), and for the sigmoid a sum, a reciprocal accurate to one unit and a product."""
    g = np.where(np.isfinite(_f64(g)), np.abs(_f64(g)), 0.0)
    return (2.0 + 0.5 * g + 2.0) * 2.0 ** -23


def scan_error(g, u, h0=None, lengths=None, form="decay"):
    """Bound of |h - exact| for every token, of an fp32 scan in any order of composition: first-order
    running error analysis.  M is the scan of magnitudes, which bounds every intermediate value of
    a composition of maps h -> A h + H; a token's gate error e enters as e (a M_{t-1} + |b u|), and the
    roundings that touch token t's value (its input product, its multiply-add, and one multiply-add in
    each of at most five levels of joining, applied to products of gates that round once each) as
    8 * 2^-24 M_t."""
    a, b = gates(g, form)
    with np.errstate(invalid="ignore"):
        M, _ = scan(g, np.abs(_f64(u)), None if h0 is None else np.abs(_f64(h0)), lengths, form)
    first = np.zeros((M.shape[0], 1, M.shape[2])) if h0 is None else np.abs(_f64(h0))[:, None]
    before = np.concatenate([first, M[:, :-1]], 1)
    e = gate_error(g)
    inject = e * (a * before + b * np.abs(_f64(u))) + 8 * 2.0 ** -24 * M
    batch, L, _ = M.shape
    n = _lengths(lengths, batch, L)
    E = np.zeros_like(M)
    run = np.zeros_like(M[:, 0]) if L else None
    for t in range(L):
        on = t < n
        run[on] = a[on, t] * run[on] + inject[on, t]
        E[on, t] = run[on]
    return E, M


def backward_error(g, u, y, dy, h0=None, dh_final=None, lengths=None, form="decay", h_error=None):
    """Bounds of |dg - exact|, |du - exact|, |dh0 - exact| for gradients formed in fp32 from the given y,
    before the rounding of the outputs: c is a scan from the last token to the first with gates a
    and inputs a dy, so scan_error's argument holds for it.  h_error: bounds of |h_t - y_t| where the gradients are
    formed from states h in place of y (the scan's fp32 states against its exact ones); it enters dg once,
    by c b, whose own error changes it by less than 2^-10 of it."""
    a, b = gates(g, form)
    y, dy, u = _f64(y), _f64(dy), None if u is None else _f64(u)
    batch, L, D = y.shape
    n = _lengths(lengths, batch, L)
    start = np.zeros((batch, D)) if h0 is None else _f64(h0)
    M = np.zeros((batch, D)) if dh_final is None else np.abs(_f64(dh_final))
    E = np.zeros((batch, D))
    e, r = gate_error(g), 2.0 ** -24
    Eg, Eu = np.zeros_like(y), np.zeros_like(y)
    for t in reversed(range(L)):
        on = t < n
        G, EG = np.abs(dy[on, t]) + M[on], E[on] + r * (np.abs(dy[on, t]) + M[on])
        M[on] = a[on, t] * G
        E[on] = a[on, t] * EG + (e[on, t] + 8 * r) * M[on]
        before = np.abs((y[:, t - 1] if t else start)[on])
        if form == "decay":
            Eu[on, t] = EG
            Eg[on, t] = (E[on] + 2 * r * M[on]) * before
        else:
            span = before + np.abs(u[on, t])
            Eu[on, t] = b[on, t] * EG + (e[on, t] + r) * b[on, t] * G
            Eg[on, t] = b[on, t] * span * (E[on] + (e[on, t] + 4 * r) * M[on])
        if h_error is not None and t:
            Eg[on, t] += (1 + 2.0 ** -10) * M[on] * b[on, t] * h_error[on, t - 1]
    return Eg, Eu, E


def quantize_rows(x):
    """(q, scale) of the row quantiser in the fp32 arithmetic that defines it."""
    x = np.asarray(_f64(x), np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.max(np.abs(x), axis=-1)
        scale = np.maximum(amax * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126)).astype(np.float32)
        ok = np.isfinite(x).all(axis=-1)
        scale = np.where(ok, scale, np.float32(np.nan))
        q = np.rint(x * (np.float32(1) / scale)[..., None])
        q = np.where(ok[..., None], q, 0).astype(np.int8)
    return q, scale


def matmul_i8(q, q_scale, w, w_scale, bias=None):
    """The scaled product in fp64 (exact integer sums)."""
    s = np.asarray(q, np.int64) @ np.asarray(w, np.int64).T if np.asarray(q).size < 1 << 16 else \
        np.asarray(q, np.float64) @ np.asarray(w, np.float64).T   # sums below 2^53: exact as well
    out = s * _f64(q_scale)[..., None] * _f64(w_scale)
    return out if bias is None else out + _f64(bias)

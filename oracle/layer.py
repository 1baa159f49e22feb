"""fp64 oracle of what surrounds the recurrence in its layer: the short causal convolution and the root-mean-square
norm with their gradients, and the activations (numpy, from the definitions; shares no code with the GPU path), with
bounds of the fp32 kernels' errors.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24   # half a unit of fp32, relative


def _f64(t):
    return np.asarray(t.detach().double().cpu().numpy() if hasattr(t, "detach") else t, np.float64)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def activate(v, act):
    if act == "silu":
        return v * sigmoid(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


def sigmoid_error(v):
    """Relative error of a sigmoid formed in fp32 as 1 / (1 + 2^(-v log2 e)): the exponent's two roundings
    (|v| 2^-24 each, relative to e^-v), an exponential and a reciprocal of one unit (2^-23) each, a sum; the
    exponential's error enters by its share 1 - g of the sum."""
    return (2 * np.abs(v) + 2) * U * sigmoid(-v) + 3 * U


def activate_error(v, e_v, act):
    """Bound of |act(v') - act(v)| for a v' within e_v of v, activated in fp32."""
    if act == "silu":   # |silu'| < 1.1; the product rounds once
        return 1.1 * e_v + np.abs(activate(v, act)) * (sigmoid_error(v) + U) + 1e-36
    if act == "gelu_tanh":
        # the sigmoid's argument a = 1.6 (v + 0.045 v^3) rounds five times: 5 |a| u relative to e^-a; |gelu'| < 1.2
        a = np.sqrt(8.0 / np.pi) * (np.abs(v) + 0.044715 * np.abs(v) ** 3)
        near = sigmoid(-np.sqrt(8.0 / np.pi) * (v + 0.044715 * v ** 3))
        return 1.2 * e_v + np.abs(activate(v, act)) * ((7 * a + 2) * U * near + 4 * U) + 1e-36
    return e_v


def _lengths(lengths, batch, L):
    return np.full(batch, L) if lengths is None else np.clip(np.asarray(_f64(lengths), np.int64), 0, L)


def _past(x, state, W):
    """Every sequence's starting state and tokens in one array."""
    first = np.zeros((x.shape[0], W - 1, x.shape[2])) if state is None else _f64(state)
    return np.concatenate([first, x], 1)


def conv(x, w, bias=None, state=None, lengths=None, act="silu"):
    """(y, state_out, bound of |y - exact| before y's rounding)."""
    x, w = _f64(x), _f64(w)
    batch, L, D = x.shape
    W, n = w.shape[1], _lengths(lengths, batch, L)
    past = _past(x, state, W)
    b = np.zeros(D) if bias is None else _f64(bias)
    y, err = np.zeros_like(x), np.zeros_like(x)
    out = np.zeros((batch, W - 1, D))
    for i in range(batch):
        for t in range(n[i]):
            v = b + sum(w[:, k] * past[i, t + k] for k in range(W))
            size = np.abs(b) + sum(np.abs(w[:, k] * past[i, t + k]) for k in range(W))
            y[i, t] = activate(v, act)
            err[i, t] = activate_error(v, (W + 1) * U * size, act)
        out[i] = past[i, n[i]:n[i] + W - 1]
    return y, out, err


def conv_backward(x, w, dy, bias=None, state=None, dstate_out=None, lengths=None, act="silu"):
    """({dx, dw, dbias, dstate}, bounds of their errors before the rounding of dx and dstate)."""
    x, w, dy = _f64(x), _f64(w), _f64(dy)
    batch, L, D = x.shape
    W, n = w.shape[1], _lengths(lengths, batch, L)
    past = _past(x, state, W)
    b = np.zeros(D) if bias is None else _f64(bias)
    de, e_de = np.zeros_like(past), np.zeros_like(past)
    dw, db = np.zeros((D, W)), np.zeros(D)
    e_dw, e_db = np.zeros((D, W)), np.zeros(D)
    # a sum over tokens rounds at most once a token and, over the shares of work-groups, less than that again; runs
    # have at most 128 tokens, work-groups 256 runs, and a quarter of the shares is summed one by one
    chain = min(n.sum(), 128 + 256 + 2 + n.sum() // 8) * U
    for i in range(batch):
        for t in range(n[i]):
            v = b + sum(w[:, k] * past[i, t + k] for k in range(W))
            size = np.abs(b) + sum(np.abs(w[:, k] * past[i, t + k]) for k in range(W))
            if act == "silu":
                g, h = sigmoid(v), sigmoid(-v)
                slope = g * (1 + v * h)
                e_g = sigmoid_error(v)
                # 1 - g is off by g e_g + u, the multiply-add rounds once, the product once; |silu''| <= 0.5
                e_s = 0.5 * (W + 1) * U * size + np.abs(slope) * (e_g + U) + \
                    g * (np.abs(v) * (g * e_g + U) + U * (1 + np.abs(v) * h))
            else:
                slope, e_s = np.ones(D), np.zeros(D)
            z = dy[i, t] * slope
            e_z = np.abs(dy[i, t]) * e_s + U * np.abs(z)
            db += z
            e_db += e_z + chain * np.abs(z)
            for k in range(W):
                de[i, t + k] += w[:, k] * z
                e_de[i, t + k] += np.abs(w[:, k]) * (e_z + (W + 1) * U * np.abs(z))
                dw[:, k] += z * past[i, t + k]
                e_dw[:, k] += np.abs(past[i, t + k]) * (e_z + (chain + U) * np.abs(z))
        if dstate_out is not None:
            add = _f64(dstate_out)[i]
            de[i, n[i]:n[i] + W - 1] += add
            e_de[i, n[i]:n[i] + W - 1] += U * (np.abs(add) + np.abs(de[i, n[i]:n[i] + W - 1]))
    dx, e_dx = de[:, W - 1:].copy(), e_de[:, W - 1:].copy()
    dstate, e_ds = de[:, :W - 1].copy(), e_de[:, :W - 1].copy()
    for i in range(batch):   # tokens of the padding have no gradient
        dx[i, n[i]:] = 0
        e_dx[i, n[i]:] = 0
    return dict(dx=dx, dw=dw, dbias=db, dstate=dstate), dict(dx=e_dx, dw=e_dw, dbias=e_db, dstate=e_ds)


def rms_norm(total, gain, eps):
    """(y, bound of |y - exact| before y's rounding) of rows of total.  The sum of squares is of one sign, so its
    relative error is that of its additions: at most 32 in a thread, a dozen joining them (up to 2^14 for rows that
    are taken element by element, K / 64 in a thread); the root halves it, the reciprocal root is good to one unit
    (2^-23), and two products round."""
    t, g = _f64(total), _f64(gain)
    K = t.shape[-1]
    r = 1.0 / np.sqrt((t ** 2).mean(-1, keepdims=True) + eps)
    y = t * g * r
    adds = min(K, 64 + K // 64)
    return y, np.abs(y) * ((adds + 4) / 2 + 2 + 2) * U + 1e-37


def rms_norm_backward(total, gain, dy, dtotal, eps):
    """(dx, dgain, bounds of their errors before dx's rounding)."""
    t, g, dy = _f64(total), _f64(gain), _f64(dy)
    K, rows = t.shape[-1], int(np.prod(t.shape[:-1]))
    r = 1.0 / np.sqrt((t ** 2).mean(-1, keepdims=True) + eps)
    n, v = t * r, dy * g
    mean = (v * n).mean(-1, keepdims=True)
    dx = r * (v - n * mean)
    e_r = ((min(K, 64 + K // 64) + 4) / 2 + 2) * U   # relative, as above
    size = np.abs(v * n).mean(-1, keepdims=True)
    e_mean = size * ((min(K, 64 + K // 64) + 4) * U + 2 * e_r)
    part = np.abs(v) + np.abs(n * mean)
    e_dx = r * (part * (e_r + 4 * U) + np.abs(n) * e_mean)
    if dtotal is not None:
        add = _f64(dtotal)
        dx = dx + add
        e_dx = e_dx + U * (np.abs(add) + np.abs(dx))
    terms = np.abs(dy * n).reshape(rows, K)
    dgain = (dy * n).reshape(rows, K).sum(0)
    # one addition a row of a work-group, of which there are 256 at least where rows are many (taken two at a time), and
    # over the work-groups, at most 1024, a sixteenth of them and sixteen
    chain = min(rows, -(-rows // 256) + 2 + 1024 // 16 + 16)
    e_gain = terms.sum(0) * ((e_r + 2 * U) + chain * U)
    return dx, dgain, e_dx, e_gain


def matmul_i8(q, q_scale, w, w_scale, bias=None, act="none", residual=None):
    """(out, bound of |out - exact| before the output's rounding): the integer sum is exact and rounds once, two
    scale products and the bias sum round once each, the residual's sum once."""
    s = (np.asarray(q, np.float64) @ np.asarray(w, np.float64).T) * _f64(q_scale)[..., None] * _f64(w_scale)
    v = s if bias is None else s + _f64(bias)
    e = 3 * U * np.abs(s) + U * np.abs(v)
    out = activate(v, act)
    e = activate_error(v, e, act)
    if residual is not None:
        out = out + _f64(residual)
        e = e + U * (np.abs(out) + e)
    return out, e

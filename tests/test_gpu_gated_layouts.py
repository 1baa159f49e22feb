"""The gated scan's layouts (strips of 16, 32 and 64 lanes, cut or not, with and without the non-temporal hint, one or
two bf16 channels a lane) with padded batches, strided rows, far rows and sliced launches; and its gradients
against differences.  Against the fp64 oracle's bounds (oracle/gated.py), or bit for bit against a smaller call."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits, f64, say
from oracle import gated as O
from test_gpu_gated_scan import assert_within, check, half_step, make

pytestmark = pytest.mark.gpu

FORMS = ["decay", "sigmoid"]


def run(g, u, dy, h0, dh, form, lengths=None, y=None, dg=None, du=None, states=None):
    y, h = jscan.gated_scan(g, u, h0=h0, lengths=lengths, form=form, y=y, states=states)
    return (y, h, *jscan.gated_scan_backward(g, u, y, dy, h0=h0, dh_final=dh, lengths=lengths, form=form, dg=dg, du=du,
                                             states=states))


def check_against_oracle(got, g, u, dy, h0, dh, form, lengths=None):
    """(y, h, dg, du, dh0) from calls of any layout; the gradients from the given y."""
    y, h, dg, du, dh0 = got
    E, _ = O.scan_error(g, u, h0, lengths, form)
    want_y, want_h = O.scan(g, u, h0, lengths, form)
    assert_within(y, want_y, E, y.dtype, "y")
    n = np.full(g.shape[0], g.shape[1]) if lengths is None else np.clip(f64(lengths).astype(int), 0, g.shape[1])
    Eh = np.where((n > 0)[:, None], E[np.arange(len(n)), np.maximum(n, 1) - 1], 0.0)
    assert_within(h, want_h, Eh, torch.float32, "h_final")
    w = O.backward(g, u, y, dy, h0, dh, lengths, form)
    for got, a, e, t, what in zip((dg, du, dh0), w, O.backward_error(g, u, y, dy, h0, dh, lengths, form),
                                  (dg.dtype, du.dtype, torch.float32), ("dg", "du", "dh0")):
        assert_within(got, a, e, t, what)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,batch,L,D,lengths", [
    ("bf16", 1, 9001, 33, None),               # one channel a lane: narrow strips, cut
    ("bf16", 1, 4097, 2047, None),             # one channel a lane: wide strips, cut
    ("bf16", 3, 700, 2001, [700, 333, 0]),     # one channel a lane, padded
    ("bf16", 3, 700, 4000, [700, 333, 650]),   # 32 lanes, padded
    ("bf16", 3, 701, 4000, None),              # 32 lanes
    ("bf16", 2, 9000, 2048, [8191, 4500]),     # wide strips, cut: segments that are skipped or partly padding
    ("f32", 2, 6000, 1024, [5999, 10]),
])
def test_layouts_match_the_oracle(dtype, batch, L, D, lengths, form):
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    check(*make(batch, L, D, dtype, form, 3 * L + D), form, n)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,repeats,L,D", [
    ("bf16", 260, 1030, 255), ("bf16", 260, 1030, 256), ("f32", 130, 1030, 256),   # 32 lanes, the even ones with the hint
    ("bf16", 260, 400, 255), ("bf16", 260, 700, 256), ("f32", 130, 500, 256),      # 64 lanes
])
def test_padded_batches_that_fill_the_chip(dtype, repeats, L, D, form):
    """g and u as the halves of one buffer, y and the gradients as columns of wider ones; two sequences of unequal
    length against the oracle, repeated; every repetition has the same bits, and nothing is written beside."""
    args = make(2, L, D, dtype, form, 7 * L + D)
    n = torch.tensor([L - 5, L // 3], dtype=torch.int32).cuda()
    g, u, dy, h0, dh = [t.repeat(repeats, *[1] * (t.dim() - 1)) for t in args]
    proj = torch.cat([g, u], -1)
    out, grads = torch.full_like(proj, 7.0), torch.full_like(proj, 7.0)
    got = run(proj[..., :D], proj[..., D:], dy, h0, dh, form, n.repeat(repeats), y=out[..., D:], dg=grads[..., :D],
              du=grads[..., D:])
    assert (out[..., :D] == 7.0).all()
    for t in got:
        t = t.contiguous().view(repeats, -1)
        assert (t == t[:1]).all()
    check_against_oracle([t[:2].contiguous() for t in got], *args, form, n)


@pytest.mark.parametrize("form", FORMS)
def test_cut_sequence_beyond_the_cache_from_halves(form):
    """Segments of a padded sequence with the non-temporal hint, g and u the halves of one buffer."""
    L, D = 45001, 1024
    args = make(1, L, D, "bf16", form, 5)
    n = torch.tensor([L - 1001], dtype=torch.int32).cuda()
    proj, grads = torch.cat(args[:2], -1), torch.empty(1, L, 2 * D, dtype=torch.bfloat16, device="cuda")
    got = run(proj[..., :D], proj[..., D:], *args[2:], form, n, dg=grads[..., :D], du=grads[..., D:])
    say(f"{form}: ran")
    check_against_oracle(got, *args, form, n)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,D,pad", [(700, 66, 0), (700, 66, 2), (9000, 128, 2), (300, 1000, 4)])
def test_strided_halves_give_the_bits_of_contiguous_tensors(L, D, pad, form):
    """Where both start on 4 bytes and hold an even number of channels, so that one layout serves both."""
    args = make(2, L, D, "bf16", form, 22)
    want = run(*args, form)
    wide = torch.full((2, L, 2 * D + 3 * pad), 9.0, dtype=torch.bfloat16, device="cuda")
    lo, hi = slice(pad, pad + D), slice(D + 2 * pad, 2 * D + 2 * pad)
    wide[..., lo], wide[..., hi] = args[:2]
    out, grads = torch.full_like(wide, 7.0), torch.full_like(wide, 7.0)
    got = run(wide[..., lo], wide[..., hi], *args[2:], form, y=out[..., hi], dg=grads[..., lo], du=grads[..., hi])
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    check_against_oracle(got, *args, form)


@pytest.mark.parametrize("off", [-8, 0, 8])
@pytest.mark.parametrize("form", FORMS)
def test_rows_at_the_edge_of_32_bit_lane_offsets(off, form):
    """Rows of 64 MiB and a little less or more: the strips' lane offsets over three runs of rows fit 32 bits up to there,
    beyond it only wide strips are used."""
    L, D, ld = 300, 72, (1 << 25) + off
    args = make(1, L, D, "bf16", form, 29)
    buf = torch.empty((1, L, ld), dtype=torch.bfloat16, device="cuda")
    at = [slice(k, k + D) for k in (0, ld // 2 & ~1, ld // 2 + 2 * D & ~1, ld - 4 * D, ld - 2 * D, ld - D)]
    for s, t in zip(at, args[:3]):
        buf[..., s] = t
    views = [buf[..., s] for s in at]
    states = jscan.gated_scan_states(args[0])
    for keep in (None, states):
        got = run(*views[:3], *args[3:], form, y=views[3], dg=views[4], du=views[5], states=keep)
        for s, t in zip(at, args[:3]):
            assert torch.equal(bits(buf[..., s]), bits(t))
        if keep is None:
            check_against_oracle(got, *args, form)
            dg = f64(got[2])
    # from the states, dg differs by y's rounding: 2^-8 |c (1 - a) h|, half a step of each, and the fp32 bound of each
    given = (*args[:2], got[0], *args[2:], None, form)
    c, b = np.abs(O.backward(*given)[3]), O.gates(args[0], form)[1]
    before = np.abs(np.concatenate([f64(args[3])[:, None], f64(got[0])[:, :-1]], 1))
    fp32 = 2 * O.backward_error(*given, h_error=O.scan_error(*args[:2], args[3], None, form)[0])[0]
    a = f64(got[2])
    assert (np.abs(a - dg) <= 2.0 ** -8 * (1.01 * c * b * before + np.abs(a) + np.abs(dg)) + 1.01 * fp32).all()


@pytest.mark.parametrize("form", FORMS)
def test_longer_sequences_than_one_launch_counts(form):
    """2^20 sequences of two tokens and an odd number of channels need more work-items than a launch's 2^32: the scan, its
    states and both backward passes, every sequence against the same one alone."""
    batch, D = 1 << 20, 4099
    small = make(1024, 2, D, "bf16", form, 63)
    n = torch.tensor([k % 3 for k in range(1024)], dtype=torch.int32).cuda()
    g, u, dy, h0, dh = [t.repeat(batch // 1024, *[1] * (t.dim() - 1)) for t in small]
    lengths = n.repeat(batch // 1024)
    states = torch.zeros(batch, 1, D, device="cuda")
    want_states = torch.zeros(1024, 1, D, device="cuda")
    y, h = jscan.gated_scan(g, u, h0=h0, h_final=h0, lengths=lengths, form=form, states=states)
    want_y, want_h = jscan.gated_scan(*small[:2], h0=small[3], lengths=n, form=form, states=want_states)

    def same(got, want):
        for b in range(0, batch, 1024):
            assert torch.equal(got[b:b + 1024], want), b

    same(y, want_y), same(h, want_h), same(states, want_states)
    say("scan equal")
    want = jscan.gated_scan_backward(*small[:2], None, small[2], dh_final=small[4], lengths=n, form=form, states=want_states)
    got = jscan.gated_scan_backward(g, u, None, dy, dh_final=dh, dh0=h0, lengths=lengths, form=form, states=states)
    for a, b in zip(got, want):
        same(a, b)
    say("backward from states equal")
    want = jscan.gated_scan_backward(*small[:2], want_y, small[2], dh_final=small[4], lengths=n, form=form)
    got = jscan.gated_scan_backward(g, u, y, dy, dh_final=dh, dh0=dh, lengths=lengths, form=form, dg=got[0], du=got[1])
    for a, b in zip(got, want):
        same(a, b)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mean", [0.0, 3.0])
def test_gradients_against_differences(dtype, mean, form):
    """The directional derivative along the sign of each gradient, where no term cancels another, against central
    differences of the exact recurrence in fp64.  The gradient is off by the sum of its elements' bounds: the
    oracle's, and half a step of the output type of each.  A step of 1e-6 on every one of a token's up to 260
    gates moves their product by 2.6e-4, so the differences are off by (2.6e-4)^2 / 6 = 1.1e-8 of the terms'
    magnitudes from the third order and by 260 * 2^-52 / 1e-6 = 5.8e-8 of them from fp64's rounding: together
    1.2 * 2^-24, of which every element's bound holds at least one; so three bounds in all."""
    g, u, dy, h0, dh = make(2, 260, 40, dtype, form, 53)
    u = (u.float() * (0.1 if mean else 1.0) + mean).to(u.dtype)
    lengths = torch.tensor([260, 131], dtype=torch.int32).cuda()
    y, h, dg, du, dh0 = run(g, u, dy, h0, dh, form, lengths, states=jscan.gated_scan_states(g))
    p = [f64(t) for t in (g, u, h0)]
    wy, wh, exact = f64(dy), f64(dh), O.scan(g, u, h0, lengths, form)[0]
    error = O.backward_error(g, u, exact, dy, h0, dh, lengths, form, h_error=O.scan_error(g, u, h0, lengths, form)[0])

    def loss(g, u, h0):
        y, h = O.scan(g, u, h0, lengths, form)
        return (y * wy).sum() + (h * wh).sum()

    for k, got in enumerate((dg, du, dh0)):
        grad, eps = f64(got), 1e-6
        v = np.sign(grad)
        up, down = list(p), list(p)
        up[k], down[k] = p[k] + eps * v, p[k] - eps * v
        numeric, total = (loss(*up) - loss(*down)) / (2 * eps), np.abs(grad).sum()
        half = half_step(got.dtype) * np.abs(grad).sum() * (1 + 2.0 ** -7)
        say(f"{form} {dtype} mean {mean} argument {k}: {total:.8g} against {numeric:.8g}")
        assert abs(numeric - total) <= 3 * error[k].sum() + half

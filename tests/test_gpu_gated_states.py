"""bf16 gradients of the gated recurrence from saved fp32 states, against the fp64 gradients of the unrounded
recurrence (the oracle's own states, not the kernel's rounded y).

Tolerances: the oracle's running error analysis with the bound of the scan's fp32 states in place of y's
rounding (oracle/gated.py), element by element, and half a step of the output type of the value."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits, f64, say
from oracle import gated as O
from test_gpu_gated_scan import assert_within, make

pytestmark = pytest.mark.gpu

FORMS = ["decay", "sigmoid"]


def train(g, u, dy, h0, dh, form, lengths=None, states=None, **out):
    states = jscan.gated_scan_states(g) if states is None else states
    y, h = jscan.gated_scan(g, u, h0=h0, lengths=lengths, form=form, states=states)
    return (y, h, states,
            *jscan.gated_scan_backward(g, u, None, dy, dh_final=dh, lengths=lengths, form=form, states=states, **out))


def check(got, g, u, dy, h0, dh, form, lengths=None):
    """(y, h, states, dg, du, dh0) against the recurrence and its gradients without any rounding."""
    y, h, states, dg, du, dh0 = got
    batch, L, D = g.shape
    want_y, want_h = O.scan(g, u, h0, lengths, form)
    E, _ = O.scan_error(g, u, h0, lengths, form)
    assert_within(y, want_y, E, y.dtype, "y")
    n = np.full(batch, L) if lengths is None else np.clip(f64(lengths).astype(int), 0, L)
    start = np.zeros((batch, D)) if h0 is None else f64(h0)
    for b in range(batch):
        last = int(n[b])
        assert_within(h[b], want_h[b], E[b, last - 1] if last else 0.0, torch.float32, f"h_final {b}")
        rows = -(-last // 8)
        before = np.concatenate([start[b][None], want_y[b, 7::8]])[:rows]
        error = np.concatenate([np.zeros((1, D)), E[b, 7::8]])[:rows]
        assert_within(states[b, :rows], before, error, torch.float32, f"states {b}")
    args = (g, u, want_y, dy, h0, dh, lengths, form)
    dg_w, du_w, dh0_w, _ = O.backward(*args)
    Eg, Eu, E0 = O.backward_error(*args, h_error=E)
    assert_within(dg, dg_w, Eg, dg.dtype, "dg")
    assert_within(du, du_w, Eu, du.dtype, "du")
    assert_within(dh0, dh0_w, E0, torch.float32, "dh0")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("batch,L,D", [
    (1, 1, 1), (1, 2, 3), (2, 7, 40), (2, 8, 64), (5, 9, 33), (3, 16, 130), (2, 17, 33), (2, 27, 66), (1, 31, 127),
    (1, 64, 128), (2, 65, 129), (2, 130, 72), (1, 255, 66), (1, 256, 32), (2, 257, 31), (1, 263, 8), (1, 300, 1000),
    (40, 5, 1024), (300, 3, 260), (260, 29, 256), (1, 1025, 96), (1, 1000, 8194), (3, 700, 4000), (1, 2049, 2048),
    (1, 4097, 2047), (1, 9001, 33), (2, 6001, 250), (1, 20000, 64), (1, 8192, 64),
])
def test_gradients_of_the_unrounded_recurrence(batch, L, D, form):
    args = make(batch, L, D, "bf16", form, 77 * L + D)
    got = train(*args, form)
    check(got, *args, form)
    y, h = jscan.gated_scan(args[0], args[1], h0=args[3], form=form)   # keeping the states changes nothing else
    assert torch.equal(bits(y), bits(got[0])) and torch.equal(bits(h), bits(got[1]))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,D,mean,spread", [(512, 64, 3.0, 0.1), (512, 64, 1.0, 0.01), (700, 33, -5.0, 0.5), (5000, 64, 3.0, 0.1)])
def test_inputs_close_to_the_state(L, D, mean, spread, form):
    """Inputs with a mean, where h - u cancels: from y rounded to bf16 most of the sigmoid form's dg would be off by more
    than the tolerance here, which has no term of that rounding."""
    g, u, dy, h0, dh = make(2, L, D, "bf16", form, L + D)
    u = (mean + spread * u.float()).to(u.dtype)
    got = train(g, u, dy, h0, dh, form)
    check(got, g, u, dy, h0, dh, form)
    want = O.backward(g, u, O.scan(g, u, h0, None, form)[0], dy, h0, dh, None, form)[0]
    rounded = f64(jscan.gated_scan_backward(g, u, got[0], dy, h0=h0, dh_final=dh, form=form)[0])
    off = [np.linalg.norm(v - want) / np.linalg.norm(want) for v in (f64(got[3]), rounded)]
    say(f"{form} mean {mean}: dg off by {off[0]:.2e} from states, {off[1]:.2e} from y")
    assert off[0] <= 2.0 ** -8


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("batch,L,D,lengths", [
    (4, 20, 40, [0, 1, 20, 7]), (3, 513, 66, [512, 0, 513]), (2, 9000, 64, [8191, 4500]), (2, 9000, 2048, [8191, 4500]),
    (3, 3000, 25, [2999, 1, 0]), (2, 300, 31, [-5, 1000]), (70, 33, 128, None), (1, 5000, 16, [0]), (9, 64, 128, None),
    (2, 4096, 512, [4090, 4095]), (2, 900, 4000, [889, 650]),
])
def test_padded_batches(batch, L, D, lengths, form):
    """Padding holds NaN in every input and is neither read nor left unwritten; rows of states behind a sequence's last
    token are left as they were."""
    g, u, dy, h0, dh = make(batch, L, D, "bf16", form, 3 * L + D)
    n = torch.tensor([(7 * b) % (L + 1) for b in range(batch)] if lengths is None else lengths, dtype=torch.int32).cuda()
    clean = [t.clone() for t in (g, u, dy)]
    for b in range(batch):
        for t in (g, u, dy):
            t[b, max(0, min(L, int(n[b]))):] = float("nan")
    states = jscan.gated_scan_states(g).fill_(9.0)
    got = train(g, u, dy, h0, dh, form, n, states)
    for b in range(batch):
        assert (states[b, -(-max(0, min(L, int(n[b]))) // 8):] == 9.0).all()
    check(got, *clean, h0, dh, form, n)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("repeats,L,D", [(260, 400, 256), (520, 1030, 64), (40, 1100, 514), (260, 61, 256), (130, 251, 250),
                                         (130, 251, 255), (300, 1030, 255)])
def test_many_sequences(repeats, L, D, form):
    """Batches that fill the chip, the larger ones beyond the last-level cache: two sequences of unequal length against
    the oracle, repeated; every repetition has the same bits."""
    args = make(2, L, D, "bf16", form, 9 * L + D)
    n = torch.tensor([L - 3, L // 2], dtype=torch.int32).cuda()
    many = [t.repeat(repeats, *[1] * (t.dim() - 1)) for t in args]
    states = jscan.gated_scan_states(many[0]).zero_()
    got = train(*many, form, n.repeat(repeats), states)
    for t in got:
        b = bits(t).view(repeats, -1)
        assert (b == b[:1]).all()
    check([t[:2] for t in got], *args, form, n)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L,D,pad", [(700, 66, 0), (700, 33, 1), (3001, 50, 6), (9000, 128, 2)])
def test_strided_halves_and_guard_columns(L, D, pad, form):
    args = make(2, L, D, "bf16", form, 21)
    g, u, dy = args[:3]
    wide = torch.full((2, L, 2 * D + 3 * pad), 9.0, dtype=g.dtype, device="cuda")
    lo, hi = slice(pad, pad + D), slice(D + 2 * pad, 2 * D + 2 * pad)
    wide[..., lo], wide[..., hi] = g, u
    grads = torch.full_like(wide, 7.0)
    got = train(wide[..., lo], wide[..., hi], dy, args[3], args[4], form, dg=grads[..., lo], du=grads[..., hi])
    check(got, *args, form)
    keep = torch.ones(wide.shape[-1], dtype=torch.bool, device="cuda")
    keep[lo] = keep[hi] = False
    assert (grads[..., keep] == 7.0).all() and (wide[..., keep] == 9.0).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L", [0, 1, 40, 6000])
def test_states_in_place_and_no_starting_state(L, form):
    """h_final over h0 and dh0 over dh_final; without h0 and dh_final they count as zero."""
    g, u, dy, h0, dh = make(2, L, 40, "bf16", form, 8)
    want = train(g, u, dy, h0, dh, form)
    s, ds, states = h0.clone(), dh.clone(), jscan.gated_scan_states(g)
    y, h = jscan.gated_scan(g, u, h0=s, h_final=s, form=form, states=states)
    dg, du, dh0 = jscan.gated_scan_backward(g, u, None, dy, dh_final=ds, dh0=ds, form=form, states=states)
    for a, b in zip(want, (y, s, states, dg, du, ds)):
        assert torch.equal(bits(a), bits(b))
    for a, b in zip(train(g, u, dy, None, None, form), train(g, u, dy, torch.zeros_like(h0), torch.zeros_like(h0), form)):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("form", FORMS)
def test_infinite_and_extreme_gates(form):
    """-inf and the type's lowest value drop the state exactly, in the state that is walked up too."""
    g, u, dy, h0, dh = make(2, 400, 24, "bf16", form, 31)
    g[0, 100], g[0, 250, ::2], g[1, 0] = -float("inf"), torch.finfo(g.dtype).min, torch.finfo(g.dtype).min
    if form == "sigmoid":
        g[1, 50:60], g[1, 300] = float("inf"), torch.finfo(g.dtype).max
    got = train(g, u, dy, h0, dh, form)
    check(got, g, u, dy, h0, dh, form)
    assert not got[5][1].any() and not got[3][0, 100].any() and not got[3][1, 0].any()


@pytest.mark.parametrize("batch,L,D", [(2, 130, 72), (1, 20001, 64)])
def test_captured_and_replayed(batch, L, D):
    args = make(batch, L, D, "bf16", "sigmoid", 23)
    eager = train(*args, "sigmoid")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(*args, "sigmoid")
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train(*args, "sigmoid")
    for replay in range(4):
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        again = train(*args, "sigmoid")
        torch.cuda.synchronize()
        for a, b, c in zip(out, eager, again):
            assert torch.equal(bits(a), bits(b)) and torch.equal(bits(a), bits(c)), f"replay {replay}"


def test_fp32_keeps_no_states_and_refusals():
    g, u, dy, h0, dh = make(2, 20, 8, "bf16", "decay", 1)
    assert jscan.gated_scan_states(g.float()) is None and jscan.gated_scan_states(g).shape == (2, 3, 8)
    states = jscan.gated_scan_states(g)
    y, _ = jscan.gated_scan(g, u, states=states)
    for kw in (dict(states=states[:, :2]), dict(states=states.bfloat16()), dict(states=states.cpu()),
               dict(g=g.float(), u=u.float(), states=states)):
        with pytest.raises(ValueError):
            jscan.gated_scan(**{**dict(g=g, u=u), **kw})
    for kw in (dict(u=None), dict(states=None, y=None), dict(states=states[:1]), dict(dy=dy.float())):
        with pytest.raises(ValueError):
            jscan.gated_scan_backward(**{**dict(g=g, u=u, y=None, dy=dy, states=states), **kw})
    with pytest.raises(jscan.JScanError):   # the states over an input
        jscan.gated_scan_backward(g, u, None, dy, dh0=states.view(-1)[:16].view(2, 8), states=states)

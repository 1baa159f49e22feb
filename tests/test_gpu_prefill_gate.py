"""The selective scan with its skip and output gate on the GPU: states bit for bit those of the scan without
them, outputs against the definition in fp64.

Tolerance of the outputs, given the scan's own y (which other tests hold against the oracle): in fp32 the gated call forms
the same fp32 y, so what is left is the skip's multiply-add (2^-24 of its result), the gate's sigmoid and its product as
the oracle bounds them, the product with y (2^-24) and half a step of the output; in bf16 the scan's y is rounded once
more on the way (half a step of it, times the gate)."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
import oracle
from gpu_util import assert_parity, bits, f64
from oracle import layer as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def inputs(batch, L, D, dtype, form="diagonal", seed=0):
    dt = DT[dtype]
    A = -torch.exp(0.5 * normal(seed + 1, D, 16)) * torch.arange(1, 17)
    if form == "complex":
        A[:, 1::2] = normal(seed + 2, D, 8)
    if form == "scalar":
        A = A[:, 0].contiguous()
    return {k: v.cuda() for k, v in dict(
        x=normal(seed + 3, batch, L, D).to(dt), delta=torch.exp(normal(seed + 4, batch, L, D) - 3).to(dt), A=A,
        B=normal(seed + 5, batch, L, 16).to(dt), C=normal(seed + 6, batch, L, 16).to(dt), skip=normal(seed + 7, D),
        z=(2 * normal(seed + 8, batch, L, D)).to(dt), h0=normal(seed + 9, batch, D, 16)).items()}


def plain(c, form, chunk=None):
    args = [c[k] for k in ("x", "delta", "A", "B", "C")]
    if chunk is not None and form == "diagonal":
        return jscan.prefill_chunked(*args, h0=c["h0"], chunk=chunk)
    return {"diagonal": jscan.prefill, "scalar": jscan.prefill_scalar_a, "complex": jscan.prefill_complex}[form](*args, h0=c["h0"])


def assert_gated(out, y, x, skip, z, what):
    """out against (y + skip x) silu(z), y the scan's output in out's type."""
    y64, x64 = f64(y), f64(x)
    sum_ = y64 if skip is None else y64 + f64(skip) * x64
    e = torch.finfo(y.dtype).eps / 2 * np.abs(y64) if y.dtype == torch.bfloat16 else np.zeros_like(y64)
    # the fp32 y that the bf16 one stands for is at most that far; the multiply-add rounds to fp32
    e = e + O.U * np.abs(sum_)
    if z is not None:
        z64 = f64(z)
        gate, e_gate = O.activate(z64, "silu"), O.activate_error(z64, 0.0, "silu")
        want = sum_ * gate
        e = e * (np.abs(gate) + e_gate) + (np.abs(sum_) * e_gate) + O.U * np.abs(want)
    else:
        want = sum_
    tol = e + torch.finfo(out.dtype).eps / 2 * (np.abs(want) + e) + 1e-36
    got = f64(out)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {tuple(np.argwhere(bad)[0])}"


SHAPES = [(1, 1, 8), (2, 3, 32), (1, 63, 64), (2, 64, 40), (1, 65, 96), (3, 128, 32), (1, 129, 256), (2, 193, 64), (1, 1000, 32),
          (4, 7, 104)]


@pytest.mark.parametrize("form", ["diagonal", "scalar", "complex"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,L,D", SHAPES)
def test_token_by_token(batch, L, D, dtype, form):
    c = inputs(batch, L, D, dtype, form, seed=L + D)
    for use_skip, use_z in ((True, True), (True, False), (False, True)):
        skip, z = c["skip"] if use_skip else None, c["z"] if use_z else None
        out, h = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=skip, z=z, h0=c["h0"], form=form)
        y, h_ref = plain(c, form)
        assert torch.equal(bits(h), bits(h_ref))
        assert_gated(out, y, c["x"], skip, z, f"skip {use_skip} z {use_z}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,L,D,chunk", [(1, 1000, 64, 100), (2, 513, 40, 64), (1, 2048, 96, 0), (3, 777, 8, 0), (1, 300, 8192, 0), (1, 17, 40, 0),
                                             (2, 3000, 24, 0), (1, 1, 8, 0), (5, 130, 1000, 0),
                                             (1, 1100, 264, 333), (2, 40, 32, 16)])
def test_time_parallel(batch, L, D, chunk, dtype):
    c = inputs(batch, L, D, dtype, seed=L)
    out, h = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=c["z"], h0=c["h0"], chunk=chunk)
    if chunk:
        y, h_ref = plain(c, "diagonal", chunk)
        assert torch.equal(bits(h), bits(h_ref))
        assert_gated(out, y, c["x"], c["skip"], c["z"], "segments")
    else:   # segments of the call's own choice, or none
        y_ref, h_ref = oracle.prefill(*(c[k].cpu() for k in ("x", "delta", "A", "B", "C")), h0=c["h0"].cpu())
        want = (y_ref + f64(c["skip"]) * f64(c["x"])) * O.activate(f64(c["z"]), "silu")
        assert_parity(f64(out), want, DT[dtype], "automatic")
        assert_parity(f64(h), h_ref, torch.float32, "state")
    for form in ("scalar", "complex"):   # automatic is token by token there
        c = inputs(batch, 130, 32, dtype, form, seed=L)
        a = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=c["z"], form=form, chunk=0)
        b = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=c["z"], form=form)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunk", [None, 100])
def test_against_the_oracle(dtype, chunk):
    c = inputs(2, 300, 64, dtype, seed=77)
    out, h = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=c["z"], h0=c["h0"], chunk=chunk)
    y_ref, h_ref = oracle.prefill(*(c[k].cpu() for k in ("x", "delta", "A", "B", "C")), h0=c["h0"].cpu())
    want = (y_ref + f64(c["skip"]) * f64(c["x"])) * O.activate(f64(c["z"]), "silu")
    assert_parity(f64(out), want, DT[dtype], "gated scan")
    assert_parity(f64(h), h_ref, torch.float32, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,wide,start", [(64, 128, 0), (64, 136, 72), (40, 80, 40)])
@pytest.mark.parametrize("chunk", [None, 64])
def test_z_as_a_slice_of_a_wider_projection(D, wide, start, chunk, dtype):
    c = inputs(2, 150, D, dtype, seed=D)
    proj = normal(5, 2, 150, wide).to(DT[dtype]).cuda()
    z = proj[..., start:start + D]
    state = c["h0"].clone()
    a = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=z, h0=state, h_final=state, chunk=chunk)
    b = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=z.contiguous(), h0=c["h0"], chunk=chunk)
    assert a[1] is state and torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))


@pytest.mark.parametrize("form", ["diagonal", "scalar", "complex"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,D", [(1, 8), (2, 64), (5, 96), (33, 40), (1, 8192)])
def test_steps(batch, D, dtype, form):
    L = 4
    c = inputs(batch, L, D, dtype, form, seed=D)
    step = {"diagonal": jscan.step, "scalar": jscan.step_scalar_a, "complex": jscan.step_complex}[form]
    proj = torch.zeros(batch, L, 2 * D, dtype=DT[dtype], device="cuda")
    proj[..., D:] = c["z"]
    h, h_ref = c["h0"].clone(), c["h0"].clone()
    wide = torch.zeros(batch, D + 8, dtype=DT[dtype], device="cuda")
    for t in range(L):
        args = [c["x"][:, t], c["delta"][:, t], c["A"], c["B"][:, t], c["C"][:, t]]
        skip, z = (c["skip"], proj[:, t, D:]) if t < 2 else (None, proj[:, t, D:]) if t == 2 else (c["skip"], None)
        out = jscan.step_gate(h, *args, skip=skip, z_t=z, form=form, y_t=wide[:, :D] if t == 1 else None)
        y = step(h_ref, *args)
        assert torch.equal(bits(h), bits(h_ref))
        assert_gated(out, y, args[0], skip, z, f"token {t}")
    assert not wide[:, D:].any()


def test_no_tokens():
    c = inputs(2, 3, 32, "f32")
    e = lambda t: t[:, :0].contiguous()   # noqa: E731
    for chunk in (None, 0, 5):
        y, h = jscan.prefill_gate(e(c["x"]), e(c["delta"]), c["A"], e(c["B"]), e(c["C"]), skip=c["skip"], z=e(c["z"]), h0=c["h0"],
                                  chunk=chunk)
        assert y.shape == (2, 0, 32) and torch.equal(h, c["h0"])
    _, h = jscan.prefill_gate(e(c["x"]), e(c["delta"]), c["A"], e(c["B"]), e(c["C"]), z=e(c["z"]))
    assert not h.any()
    empty = inputs(0, 3, 32, "f32")
    y, h = jscan.prefill_gate(*(empty[k] for k in ("x", "delta", "A", "B", "C")), skip=empty["skip"])
    assert y.shape == (0, 3, 32) and h.shape == (0, 32, 16)


def test_special_values_stay_in_their_channel():
    c = inputs(1, 100, 64, "f32", seed=3)
    args = lambda z: dict(skip=c["skip"], z=z)   # noqa: E731
    base, _ = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], **args(c["z"]))
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = c["z"].clone()
        z[0, 50, 9] = bad
        out, _ = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], **args(z))
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[0, 50, 9] = False
        assert torch.equal(out[keep], base[keep]) and not torch.isfinite(out[0, 50, 9])
    z = torch.full_like(c["z"], -200.0)   # a closed gate
    out, _ = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], **args(z))
    assert not out.any()


@pytest.mark.parametrize("D,chunk", [(64, None), (64, 0), (40, None)])
def test_captured_and_replayed_and_on_another_stream(D, chunk):
    c = inputs(1, 1200, D, "bf16", seed=4)
    n = jscan.prefill_gate_workspace_bytes(1, 1200, D, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if chunk is not None else None
    h = c["h0"].clone()

    def work():
        y, hf = jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"], z=c["z"], h0=c["h0"], chunk=chunk,
                                   workspace=ws)
        y_t = jscan.step_gate(h, c["x"][:, 5], c["delta"][:, 5], c["A"], c["B"][:, 5], c["C"][:, 5], skip=c["skip"],
                              z_t=c["z"][:, 5])
        return [y, hf, y_t]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        c["z"].copy_(normal(50 + i, 1, 1200, D))
        h.copy_(c["h0"])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        h.copy_(c["h0"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = work()
        side.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want)), f"replay {i}"

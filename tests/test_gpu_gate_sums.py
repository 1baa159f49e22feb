"""What the bf16 output of the scan with its skip and output gate is rounded from, on the GPU.

A call on bf16 tensors and one on the same values in fp32 advance the same fp32 states.  Where the sum over the states
is formed in fp32, the bf16 output is the fp32 call's output rounded once: no tolerance.  Where a token-by-token call
takes each state into the sum rounded to bf16 (half a step: 2^-8 of it at most), the two sums differ by at most 2^-8
of sum_n |C_n h_n|, and by the roundings of two fp32 sums of 16 products, 2 * 17 * 2^-24 of it; the skip's
multiply-add rounds both (2^-24 each), as do the gate's factor (the same in both) and the output (half a step).  The
states of every token come from the decode step, whose states are the scan's bit for bit."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits

pytestmark = pytest.mark.gpu

STEP = {"diagonal": jscan.step, "scalar": jscan.step_scalar_a, "complex": jscan.step_complex}


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def inputs(batch, L, D, form="diagonal", seed=0):
    """bf16 inputs and the same values in fp32."""
    A = -torch.exp(0.5 * normal(seed + 1, D, 16)) * torch.arange(1, 17)
    if form == "complex":
        A[:, 1::2] = normal(seed + 2, D, 8)
    if form == "scalar":
        A = A[:, 0].contiguous()
    typed = {k: v.bfloat16().cuda() for k, v in dict(
        x=normal(seed + 3, batch, L, D), delta=torch.exp(normal(seed + 4, batch, L, D) - 3), B=normal(seed + 5, batch, L, 16),
        C=normal(seed + 6, batch, L, 16), z=2 * normal(seed + 7, batch, L, D)).items()}
    rest = {k: v.cuda() for k, v in dict(A=A, skip=normal(seed + 8, D), h0=normal(seed + 9, batch, D, 16)).items()}
    return dict(typed, **rest), dict({k: v.float() for k, v in typed.items()}, **rest)


def gate(c, skip, z, **kw):
    return jscan.prefill_gate(c["x"], c["delta"], c["A"], c["B"], c["C"], skip=c["skip"] if skip else None, z=c["z"] if z else None,
                              h0=c["h0"], **kw)


@pytest.mark.parametrize("batch,L,D,chunk", [
    (1, 1, 32, 0), (2, 40, 32, 0), (3, 129, 96, 0), (1, 64, 64, 0), (1, 200, 8192, 0), (30, 70, 640, 0),   # token by token
    (1, 2048, 96, 0), (1, 777, 8, 0), (2, 3000, 24, 0),                                                    # segments of its choice
    (1, 300, 64, 100), (2, 77, 40, 16), (1, 130, 32, 1000),                                                # given segments
    (2, 150, 40, None), (3, 17, 8, None)])                                                                 # odd widths
def test_output_is_the_fp32_one_rounded_once(batch, L, D, chunk):
    c16, c32 = inputs(batch, L, D, seed=L + D)
    for skip, z in ((True, True), (True, False), (False, True)):
        y16, h16 = gate(c16, skip, z, chunk=chunk)
        y32, h32 = gate(c32, skip, z, chunk=chunk)
        assert torch.equal(bits(h16), bits(h32))
        off = int((bits(y16) != bits(y32.bfloat16())).sum())
        assert off == 0, f"skip {skip} z {z}: {off} of {y16.numel()} elements"


@pytest.mark.parametrize("form,chunk", [("diagonal", None), ("scalar", None), ("complex", None), ("scalar", 0), ("complex", 0)])
@pytest.mark.parametrize("batch,L,D", [(1, 1, 32), (2, 65, 64), (1, 130, 96)])
def test_states_rounded_token_by_token_stay_in_the_stated_bound(batch, L, D, form, chunk):
    c16, c32 = inputs(batch, L, D, form, seed=L)
    size, h = torch.empty(batch, L, D, dtype=torch.float64, device="cuda"), c32["h0"].clone()
    for t in range(L):
        STEP[form](h, c32["x"][:, t], c32["delta"][:, t], c32["A"], c32["B"][:, t], c32["C"][:, t])
        size[:, t] = (h.double() * c32["C"][:, t, None].double()).abs().sum(-1)
    for skip, z in ((True, True), (True, False), (False, True)):
        y16, h16 = gate(c16, skip, z, form=form, chunk=chunk)
        y32, h32 = gate(c32, skip, z, form=form, chunk=chunk)
        assert torch.equal(bits(h16), bits(h32)) and torch.equal(bits(h16), bits(h))
        want = y32.double()
        zv = c32["z"].double()
        factor = (zv * torch.sigmoid(zv)).abs() * (1 + 2.0 ** -16) if z else torch.ones_like(want)   # its fp32 error: |z| < 16
        add = size + (c32["skip"].double() * c32["x"].double()).abs() if skip else size
        e = factor * ((2.0 ** -8 + 34 * 2.0 ** -24) * size + 2 * 2.0 ** -24 * add) + 2 * 2.0 ** -24 * want.abs()
        bad = ~((y16.double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e) + 1e-36)
        assert not bad.any(), f"skip {skip} z {z}: {int(bad.sum())} of {bad.numel()}"

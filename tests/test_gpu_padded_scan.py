"""A padded batch through the convolution and the scan with its gate, on the GPU: the scan has no lengths, and a step of
zero (delta = 0 in the padding, where x, B and C are finite) leaves every state as it was.  The rows in front of the
padding are those of each sequence alone, bit for bit, and so are the states token by token.

In segments a state that the padding's segments take on goes through the maps of whole segments, h -> e^(A S) h + h_loc
with S a sum of at most 32 steps, where the sequence alone walks its last segment: e^(A S) is off by the rounding of S
and of the exponent, under 40 * 2^-24 |A S|, and each of the L tokens or maps by at most 4 roundings of 2^-24, all
relative to |h0| + sum |delta x B|, which bounds every state on the way (A < 0)."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 40])
@pytest.mark.parametrize("form,chunk", [("diagonal", None), ("diagonal", 32), ("scalar", None), ("complex", None)])
def test_a_step_of_zero_in_the_padding_keeps_the_state(form, chunk, D, dtype):
    L, lengths, W = 200, [200, 1, 64, 131, 0, 33], 4
    dt, n = DT[dtype], torch.tensor(lengths, dtype=torch.int32, device="cuda")
    batch = len(lengths)
    A = -torch.exp(0.5 * normal(1, D, 16))
    if form == "complex":
        A[:, 1::2] = normal(2, D, 8)
    A = (A[:, 0].contiguous() if form == "scalar" else A).cuda()
    x, z = (normal(i, batch, L, D).to(dt).cuda() for i in (3, 4))
    B, C = (normal(i, batch, L, 16).to(dt).cuda() for i in (5, 6))
    delta = torch.exp(normal(7, batch, L, D) - 2).to(dt).cuda()
    w, skip, h0 = (normal(8, D, W) / 2).cuda(), normal(9, D).cuda(), normal(10, batch, D, 16).cuda()
    inside = (torch.arange(L, device="cuda")[None, :] < n[:, None])[..., None]
    u, past = jscan.causal_conv(x, w, lengths=n)
    y, h = jscan.prefill_gate(u, torch.where(inside, delta, 0), A, B, C, skip=skip, z=z, h0=h0, form=form, chunk=chunk)
    _, lost = jscan.prefill_gate(u, delta, A, B, C, skip=skip, z=z, h0=h0, form=form, chunk=chunk)
    for b, t in enumerate(lengths):
        def one(v):
            return v[b:b + 1, :t].contiguous()

        u1, past1 = jscan.causal_conv(one(x), w)
        y1, h1 = jscan.prefill_gate(u1, one(delta), A, one(B), one(C), skip=skip, z=one(z), h0=h0[b:b + 1], form=form, chunk=chunk)
        assert torch.equal(bits(u[b, :t]), bits(u1[0])) and torch.equal(bits(past[b]), bits(past1[0]))
        assert torch.equal(bits(y[b, :t]), bits(y1[0]))
        if chunk is None:
            assert torch.equal(bits(h[b]), bits(h1[0]))
        else:
            d, v = one(delta)[0].double(), one(u)[0].double()
            size = h0[b].double().abs() + ((d * v).abs()[..., None] * one(B)[0].double().abs()[:, None]).sum(0)
            tol = 2.0 ** -24 * (4 * L + 40 * A.double().abs() * d.sum(0)[:, None]) * size
            assert ((h[b].double() - h1[0].double()).abs() <= tol).all()
        assert t == L or not torch.equal(bits(lost[b]), bits(h1[0]))   # what the padding's own steps make of it

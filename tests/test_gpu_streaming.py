"""Tensors larger than the last-level cache, whose kernels load and store past it: bit for bit what the calls give for
pieces that fit, channel by channel (convolution) or row by row (norm), which other tests hold against the definition.
Only the gradients that are sums over all tokens or rows are added up in another order."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def same(a, b):
    return torch.equal(bits(a.contiguous()), bits(b.contiguous()))


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype,batch,D", [("bf16", 8, 8401), ("f32", 4, 8404)])
def test_convolution(dtype, batch, D, W, padded):
    L, piece = 1001, 2000
    x, dy = (normal(i, batch, L, D).to(DT[dtype]) for i in (1, 2))
    w, bias = normal(3, D, W) / W ** 0.5, 0.3 * normal(4, D)
    state, ds = (normal(i, batch, W - 1, D).to(DT[dtype]) for i in (5, 6))
    lengths = torch.tensor([0, 1, 130, 1001, 512, 700, 64, 999][:batch], dtype=torch.int32, device="cuda") if padded else None
    assert x.numel() * x.element_size() * 2 > 256 << 20
    y, out = jscan.causal_conv(x, w, bias=bias, state=state, lengths=lengths)
    dx, dw, db, dstate = jscan.causal_conv_backward(x, w, dy, bias=bias, state=state, dstate_out=ds, lengths=lengths)
    for a in range(0, D, piece):
        cut = slice(a, min(a + piece, D))
        args = dict(bias=bias[cut], state=state[..., cut].contiguous(), lengths=lengths)
        y0, out0 = jscan.causal_conv(x[..., cut], w[cut], **args)
        assert same(y[..., cut], y0) and same(out[..., cut], out0)
        dx0, dw0, db0, dstate0 = jscan.causal_conv_backward(x[..., cut], w[cut], dy[..., cut],
                                                            dstate_out=ds[..., cut].contiguous(), **args)
        assert same(dx[..., cut], dx0) and same(dstate[..., cut], dstate0)
        # the same terms z e, added up in two orders of at most 256 additions in a chain (128 tokens of a run, then
        # runs and work-groups): 2 * 256 * 2^-24 of the sum of their sizes, and |z| <= 1.1 |dy|
        size = 1.1 * dy[..., cut].double().abs()
        if padded:
            size *= (torch.arange(L, device="cuda")[None, :] < lengths[:, None])[..., None]
        e = torch.cat([state[..., cut], x[..., cut]], 1).double().abs()
        for k in range(W):
            assert ((dw[cut, k] - dw0[:, k]).abs() <= 2.0 ** -15 * (size * e[:, k:k + L]).sum((0, 1))).all()
        assert ((db[cut] - db0).abs() <= 2.0 ** -15 * size.sum((0, 1))).all()


def test_convolution_with_its_state_in_place():
    batch, L, D = 8, 1001, 8404
    x, w, state = normal(1, batch, L, D).bfloat16(), normal(2, D, 4), normal(3, batch, 3, D).bfloat16()
    want = jscan.causal_conv(x, w, state=state)
    y, out = jscan.causal_conv(x, w, state=state, state_out=state)
    assert out is state and same(y, want[0]) and same(state, want[1])


# one, four and sixteen waves, long rows that are read again, and more rows than a launch has work-groups
@pytest.mark.parametrize("dtype,M,K", [("bf16", 70000, 500), ("bf16", 9000, 4099), ("bf16", 4000, 9008), ("bf16", 2100, 16400),
                                       ("f32", 40000, 512), ("f32", 2000, 10001), ("bf16", (1 << 20) + 77, 64)])
def test_norm(dtype, M, K):
    piece = max(1, (8 << 20) // K)
    x, res, dy, more = (normal(i, M, K).to(DT[dtype]) for i in (1, 2, 3, 4))
    gain = 1 + 0.3 * normal(5, K)
    assert x.numel() * x.element_size() * 4 > 256 << 20
    y, total = jscan.rms_norm(x, gain, residual=res)
    alone, _ = jscan.rms_norm(total, gain)
    assert same(y, alone)
    dx, dgain = jscan.rms_norm_backward(total, gain, dy, dtotal=more)
    bare, dgain_bare = jscan.rms_norm_backward(total, gain, dy)
    q, s, again = jscan.rms_norm_quantize(x, gain, residual=res) if K % 16 == 0 else (None, None, total)
    assert same(again, total)
    for a in range(0, M, piece):
        cut = slice(a, min(a + piece, M))
        y0, total0 = jscan.rms_norm(x[cut], gain, residual=res[cut])
        assert same(y[cut], y0) and same(total[cut], total0)
        assert same(dx[cut], jscan.rms_norm_backward(total0, gain, dy[cut], dtotal=more[cut])[0])
        assert same(bare[cut], jscan.rms_norm_backward(total0, gain, dy[cut])[0])
        if q is not None:
            q0, s0, _ = jscan.rms_norm_quantize(x[cut], gain, residual=res[cut])
            assert torch.equal(q[cut], q0) and same(s[cut], s0)
    # the sum's terms dy total r: r within 2^-20 of its value (its sum of K squares goes by way of lanes and waves, at
    # most 64 additions in a chain, half of whose error reaches r), and at most M / 256 + 64 additions in a chain
    want, size = torch.zeros(K, dtype=torch.float64, device="cuda"), torch.zeros(K, dtype=torch.float64, device="cuda")
    for a in range(0, M, piece):
        t, g = total[a:a + piece].double(), dy[a:a + piece].double()
        terms = g * t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)
        want += terms.sum(0)
        size += terms.abs().sum(0)
    tol = (2.0 ** -19 + (M / 256 + 64) * 2.0 ** -24) * size
    assert ((dgain - want).abs() <= tol).all() and ((dgain_bare - want).abs() <= tol).all()

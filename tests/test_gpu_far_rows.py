"""Rows so far apart that their offsets pass 2^32 elements: every call that takes a row stride gives the bits that it
gives for contiguous rows, and the rest of the buffer's rows stays as it was."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits

pytestmark = pytest.mark.gpu

ROWS, STRIDE = 140, 1 << 25   # the last row starts at 139 * 2^25 > 2^32 elements
SLOT = 8192 + 64              # columns of one operand in a row, with some behind them that no call may touch


class Far:
    """One buffer of bf16 rows; slot i of a row holds an operand."""

    def __init__(self):
        self.buf = torch.empty(ROWS * STRIDE, dtype=torch.bfloat16, device="cuda")
        self.used = self.buf.as_strided((ROWS, 8 * SLOT), (STRIDE, 1))
        self.used.fill_(7)

    def rows(self, slot, D, *lead):
        lead = lead or (ROWS,)
        strides = [STRIDE] if len(lead) == 1 else [lead[1] * STRIDE, STRIDE]
        return self.buf.as_strided((*lead, D), (*strides, 1), slot * SLOT)

    def put(self, slot, value):
        t = self.rows(slot, value.shape[-1], *value.shape[:-1])
        t.copy_(value)
        return t

    def assert_untouched(self, D):
        for slot in range(8):
            self.rows(slot, D).fill_(7)
        assert (self.used == 7).all()


@pytest.fixture(scope="module")
def far():
    f = Far()
    yield f
    del f.buf, f.used
    torch.cuda.empty_cache()


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


def same(a, b):
    return torch.equal(bits(a.contiguous()), bits(b.contiguous()))


@pytest.mark.parametrize("batch", [1, 4])
def test_convolution(far, batch):
    L, D, W = ROWS // batch, 1000, 4
    x, dy = (normal(i, batch, L, D).bfloat16() for i in (1, 2))
    w, bias, state = normal(3, D, W), normal(4, D), normal(5, batch, W - 1, D).bfloat16()
    fx, fdy = far.put(0, x), far.put(1, dy)
    y, out = jscan.causal_conv(fx, w, bias=bias, state=state, y=far.rows(2, D, batch, L))
    want = jscan.causal_conv(x, w, bias=bias, state=state)
    assert same(y, want[0]) and same(out, want[1])
    got = jscan.causal_conv_backward(fx, w, fdy, bias=bias, state=state, dx=far.rows(3, D, batch, L))
    for a, b in zip(got, jscan.causal_conv_backward(x, w, dy, bias=bias, state=state)):
        assert same(a, b)
    far.assert_untouched(D)


def test_convolution_step(far):
    D, W = 1000, 4
    x, w, bias, state = normal(1, ROWS, D).bfloat16(), normal(2, D, W), normal(3, D), normal(4, ROWS, W - 1, D).bfloat16()
    states = state.clone(), state.clone()
    y = jscan.causal_conv_step(states[0], far.put(0, x), w, bias=bias, y_t=far.rows(1, D))
    assert same(y, jscan.causal_conv_step(states[1], x, w, bias=bias)) and same(*states)
    far.assert_untouched(D)


@pytest.mark.parametrize("D,chunk", [(64, None), (64, 16), (8192, None), (8192, 32)])
def test_scan_with_gate(far, D, chunk):
    x, z = normal(1, 1, ROWS, D).bfloat16(), normal(2, 1, ROWS, D).bfloat16()
    delta, A = torch.exp(normal(3, 1, ROWS, D) - 3).bfloat16(), -torch.exp(normal(4, D, 16))
    B, C, skip = normal(5, 1, ROWS, 16).bfloat16(), normal(6, 1, ROWS, 16).bfloat16(), normal(7, D)
    got = jscan.prefill_gate(x, delta, A, B, C, skip=skip, z=far.put(0, z), chunk=chunk)
    want = jscan.prefill_gate(x, delta, A, B, C, skip=skip, z=z, chunk=chunk)
    assert same(got[0], want[0]) and same(got[1], want[1])
    far.assert_untouched(D)


def test_step_with_gate(far):
    D = 512
    x, z = normal(1, ROWS, D).bfloat16(), normal(2, ROWS, D).bfloat16()
    delta, A = torch.exp(normal(3, ROWS, D) - 3).bfloat16(), -torch.exp(normal(4, D, 16))
    B, C, skip, h = normal(5, ROWS, 16).bfloat16(), normal(6, ROWS, 16).bfloat16(), normal(7, D), normal(8, ROWS, D, 16)
    states = h.clone(), h.clone()
    y = jscan.step_gate(states[0], x, delta, A, B, C, skip=skip, z_t=far.put(0, z), y_t=far.rows(1, D))
    assert same(y, jscan.step_gate(states[1], x, delta, A, B, C, skip=skip, z_t=z)) and same(*states)
    far.assert_untouched(D)


@pytest.mark.parametrize("K", [5, 512, 4096, 8190])
def test_norm(far, K):
    x, res, dy, more = (normal(i, ROWS, K).bfloat16() for i in (1, 2, 3, 4))
    gain = normal(5, K)
    fx, fres, fdy, fmore = (far.put(i, t) for i, t in enumerate((x, res, dy, more)))
    y, total = jscan.rms_norm(fx, gain, residual=fres, y=far.rows(4, K), total=far.rows(5, K))
    want = jscan.rms_norm(x, gain, residual=res)
    assert same(y, want[0]) and same(total, want[1])
    dx, dgain = jscan.rms_norm_backward(total, gain, fdy, dtotal=fmore, dx=far.rows(6, K))
    wanted = jscan.rms_norm_backward(want[1], gain, dy, dtotal=more)
    assert same(dx, wanted[0]) and same(dgain, wanted[1])
    if K % 16 == 0:
        q, s, total = jscan.rms_norm_quantize(fx, gain, residual=fres, total=far.rows(7, K))
        q0, s0, total0 = jscan.rms_norm_quantize(x, gain, residual=res)
        assert torch.equal(q, q0) and same(s, s0) and same(total, total0)
    far.assert_untouched(K)


def test_product_with_residual(far):
    N, K = 200, 96
    gen = torch.Generator().manual_seed(1)
    q, w = (torch.randint(-128, 128, s, dtype=torch.int8, generator=gen).cuda() for s in ((ROWS, K), (N, K)))
    sq, sw, res = torch.rand(ROWS, generator=gen).cuda(), torch.rand(N, generator=gen).cuda(), normal(2, ROWS, N).bfloat16()
    want = jscan.matmul_i8(q, sq, w, sw, activation="silu", residual=res)
    out = jscan.matmul_i8(q, sq, w, sw, out=far.rows(1, N), activation="silu", residual=far.put(0, res))
    assert same(out, want)
    stream = far.rows(0, N)
    assert same(jscan.matmul_i8(q, sq, w, sw, out=stream, activation="silu", residual=stream), want)
    far.assert_untouched(N)

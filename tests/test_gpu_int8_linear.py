"""The int8 projection on the GPU: the row quantiser bit for bit against its fp32 definition, the product
against exact integer sums in fp64, and the projection feeding the gated recurrence.

Tolerance of the product: the int32 sum is exact and rounded to fp32 once, two scale products and the
bias sum round once each: 3 * 2^-24 of the scaled product and 2^-24 of the result, then half a step of the
output type (torch.finfo(dtype).eps / 2 of the value)."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits, f64, say
from oracle import gated as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def int8(M, K, seed, low=-127):
    return torch.randint(low, 128, (M, K), generator=torch.Generator().manual_seed(seed), dtype=torch.int8).cuda()


def scales(n, seed):
    return torch.exp(torch.randn(n, generator=torch.Generator().manual_seed(seed)) - 6).cuda()


def check_product(out, q, sq, w, sw, bias):
    s = (q.double() @ w.double().t()) * sq.double()[:, None] * sw.double()   # sums below 2^53: exact
    want = s if bias is None else s + bias.double()
    tol = 3 * 2.0 ** -24 * s.abs() + 2.0 ** -24 * want.abs()
    tol = tol + torch.finfo(out.dtype).eps / 2 * (want.abs() + tol) + 1e-37
    bad = ~((out.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} outside, first at {i}: {out[i].item()} against {want[i].item()}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (2, 64), (5, 80), (1, 4096), (33, 4112), (7, 8192), (300, 1024), (2, 131056),
                                 (1030, 256), (17, 8208)])
def test_quantiser_matches_its_definition(M, K, dtype):
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(M + K)) * torch.exp(torch.randn(M, 1) * 4)).to(DT[dtype])
    q, s = jscan.quantize_rows(x.cuda())
    q_ref, s_ref = O.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), s_ref) and np.array_equal(q.cpu().numpy(), q_ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantiser_special_rows(dtype):
    x = torch.randn(12, 96, generator=torch.Generator().manual_seed(1))
    x[0], x[1, 95], x[2, 0], x[3, 50] = 0, float("nan"), float("inf"), -float("inf")
    x[4] = 1e-38
    x[5] = torch.arange(96) - 48 + 0.5            # ties
    x[5, 0] = 127
    x[6] = -0.0
    x[7] = torch.finfo(DT[dtype]).max
    x[8], x[8, 17] = 0, 2.0 ** -130
    x = x.to(DT[dtype])
    q, s = jscan.quantize_rows(x.cuda())
    q_ref, s_ref = O.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), s_ref, equal_nan=True) and np.array_equal(q.cpu().numpy(), q_ref)
    w, sw = int8(40, 96, 3), scales(40, 4)
    for out_dtype in DT.values():
        out = jscan.matmul_i8(q, s, w, sw, out_dtype=out_dtype)
        assert torch.isnan(out[1:4]).all() and not torch.isnan(out[4:]).any() and not out[0].any()


@pytest.mark.parametrize("dtype,K,wide", [("bf16", 64, 72), ("bf16", 64, 65), ("f32", 80, 84), ("f32", 32, 33)])
def test_quantiser_strided_rows_and_leading_dimensions(dtype, K, wide):
    x = torch.randn(10, wide, generator=torch.Generator().manual_seed(K)).to(DT[dtype]).cuda()
    for start in (0, wide - K):
        q, s = jscan.quantize_rows(x[:, start:start + K])
        q_ref, s_ref = O.quantize_rows(x[:, start:start + K])
        assert np.array_equal(s.cpu().numpy(), s_ref) and np.array_equal(q.cpu().numpy(), q_ref)
    x3 = x[:, :K].reshape(2, 5, K)
    q3, s3 = jscan.quantize_rows(x3)
    q, s = jscan.quantize_rows(x[:, :K])
    assert q3.shape == (2, 5, K) and s3.shape == (2, 5) and torch.equal(q3.view(10, K), q) and torch.equal(s3.view(-1), s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 16, 64), (2, 17, 48), (15, 15, 80), (16, 288, 128), (17, 33, 144), (31, 100, 512), (33, 64, 1040),
    (64, 64, 4096), (65, 127, 256), (100, 288, 8192), (127, 129, 96), (128, 128, 128), (129, 257, 272), (200, 1000, 64),
    (256, 256, 256), (257, 288, 400), (300, 513, 1024), (513, 300, 176), (1, 4096, 8192), (4, 5000, 2064), (700, 1500, 640),
    (1025, 64, 16), (40, 1030, 131056),
])
@pytest.mark.parametrize("bias", [False, True])
def test_product_matches_integer_sums(M, N, K, dtype, bias):
    q, w, sq, sw = int8(M, K, M + K), int8(N, K, N + K + 1, -128), scales(M, 1), scales(N, 2)
    b = torch.randn(N, generator=torch.Generator().manual_seed(N)).cuda() if bias else None
    out = jscan.matmul_i8(q, sq, w, sw, bias=b, out_dtype=DT[dtype])
    check_product(out, q, sq, w, sw, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [   # the larger tiles, each with rows, columns and K that end inside one
    (1000, 4100, 144), (700, 2300, 272), (2500, 2600, 1552), (2049, 5000, 272), (6000, 6001, 96), (1000, 4100, 1040),
    (3900, 4090, 2064), (4096, 4090, 1040), (8200, 8301, 144), (190, 2050, 8208), (90, 3900, 2064), (100, 4097, 4112),
    (256, 2100, 4112), (777, 2111, 2064), (500, 4100, 1040),
])
def test_large_products_match_integer_sums(M, N, K, dtype):
    q, w, sq, sw = int8(M, K, M + K), int8(N, K, N + K + 1, -128), scales(M, 1), scales(N, 2)
    b = torch.randn(N, generator=torch.Generator().manual_seed(N)).cuda()
    check_product(jscan.matmul_i8(q, sq, w, sw, bias=b, out_dtype=DT[dtype]), q, sq, w, sw, b)


def test_largest_sums_do_not_wrap():
    """K at its limit with every product at 127 * 128 or 128 * 128: the int32 sums stay below 2^31."""
    K = 131056
    q, w = torch.full((20, K), -128, dtype=torch.int8).cuda(), torch.full((24, K), -128, dtype=torch.int8).cuda()
    w[1::2] = 127
    one_m, one_n = torch.ones(20).cuda(), torch.ones(24).cuda()
    out = jscan.matmul_i8(q, one_m, w, one_n, out_dtype=torch.float32)
    assert (out[:, ::2] == 128 * 128 * K).all()
    assert (out[:, 1::2].double() == float(np.float32(-127 * 128 * K))).all()


def test_output_rows_with_a_stride():
    q, w, sq, sw = int8(50, 160, 5), int8(70, 160, 6), scales(50, 1), scales(70, 2)
    want = jscan.matmul_i8(q, sq, w, sw)
    for wide, start in ((96, 8), (81, 3)):
        buf = torch.full((50, wide), 3.0, dtype=torch.bfloat16, device="cuda")
        jscan.matmul_i8(q, sq, w, sw, out=buf[:, start:start + 70])
        assert torch.equal(bits(buf[:, start:start + 70]), bits(want))
        buf[:, start:start + 70] = 3.0
        assert (buf == 3.0).all()


def test_rows_beyond_32_bit_offsets():
    """q and out of more than 2^31 bytes and elements: the far rows against the same rows alone."""
    M, K, N = (1 << 18) + 5, 8208, 8200
    q = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    q[-300:] = int8(300, K, 9)
    q[:100] = int8(100, K, 10)
    w, sq, sw = int8(N, K, 11), torch.ones(M, device="cuda"), scales(N, 2)
    out = jscan.matmul_i8(q, sq, w, sw)
    assert torch.equal(bits(out[-300:]), bits(jscan.matmul_i8(q[-300:].contiguous(), sq[:300].contiguous(), w, sw)))
    assert torch.equal(bits(out[:100]), bits(jscan.matmul_i8(q[:100].contiguous(), sq[:100].contiguous(), w, sw)))
    assert not out[100:-300].any()


def test_more_rows_than_one_grid_dimension_counts():
    """2^28 rows of 16 values, two columns: every row against its copy in a small case."""
    M, K, N = (1 << 28) + 4096, 16, 2
    x0 = torch.randn(4096, K, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    w, sw = int8(N, K, 5), scales(N, 6)
    q0, s0 = jscan.quantize_rows(x0)
    out0 = jscan.matmul_i8(q0, s0, w, sw)
    q, s = jscan.quantize_rows(x0.repeat(M // 4096, 1))
    assert (q.view(-1, 4096 * K) == q0.view(1, -1)).all() and (s.view(-1, 4096) == s0).all()
    out = jscan.matmul_i8(q, s, w, sw)
    assert (out.view(-1, 4096 * N) == out0.view(1, -1)).all()


def test_empty_sizes_write_nothing():
    w, sw = int8(8, 32, 1), scales(8, 1)
    q, s = jscan.quantize_rows(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)
    assert jscan.matmul_i8(q, s, w, sw).shape == (0, 8)
    assert jscan.matmul_i8(int8(3, 32, 1), scales(3, 1), w[:0], sw[:0]).shape == (3, 0)


@pytest.mark.parametrize("M,N,K", [(1, 640, 512), (37, 300, 4112), (600, 1500, 640), (2100, 4100, 272)])
def test_captured_and_replayed(M, N, K):
    """Quantiser and product recorded into a graph; every replay on new contents gives the eager calls' bits."""
    r = torch.Generator().manual_seed(M)
    w, sw, b = int8(N, K, 3), scales(N, 4), scales(N, 5)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        jscan.matmul_i8(*jscan.quantize_rows(x), w, sw, bias=b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = jscan.quantize_rows(x)
        out = jscan.matmul_i8(q, s, w, sw, bias=b)
    for k in range(4):
        x.copy_(torch.randn(M, K, generator=r).to(torch.bfloat16).cuda() * 2.0 ** k)
        graph.replay()
        torch.cuda.synchronize()
        q1, s1 = jscan.quantize_rows(x)
        assert torch.equal(q, q1) and torch.equal(s, s1)
        assert torch.equal(out, jscan.matmul_i8(q1, s1, w, sw, bias=b))


def test_calls_on_two_streams_at_once():
    """Layers of different sizes side by side on two streams give what they give alone."""
    layers = []
    for M, N, K in ((3000, 2100, 272), (40, 4000, 4096)):
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).cuda()
        layers.append((x, int8(N, K, N), scales(N, K)))
    alone = [jscan.matmul_i8(*jscan.quantize_rows(x), w, sw) for x, w, sw in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(6):
        for i, (x, w, sw) in enumerate(layers):
            with torch.cuda.stream(streams[i]):
                got[i].append(jscan.matmul_i8(*jscan.quantize_rows(x), w, sw))
    torch.cuda.synchronize()
    for a, outs in zip(alone, got):
        assert all(torch.equal(a, o) for o in outs)


def test_binding_refusals_on_the_gpu():
    q, w, sq, sw = int8(4, 32, 5), int8(6, 32, 6), scales(4, 1), scales(6, 2)
    for kw in (dict(q=q.float()), dict(w=w[:, :16]), dict(w=w.t()), dict(q_scale=sq[:3]), dict(w_scale=sw.double()),
               dict(bias=sq), dict(out_dtype=torch.float16), dict(out=torch.empty(4, 5, device="cuda"))):
        with pytest.raises(ValueError):
            jscan.matmul_i8(**{**dict(q=q, q_scale=sq, w=w, w_scale=sw), **kw})
    with pytest.raises(jscan.JScanError):
        jscan.quantize_rows(torch.zeros(2, 40, device="cuda"))
    with pytest.raises(ValueError):
        jscan.quantize_rows(torch.zeros(2, 32, device="cuda", dtype=torch.float16))


@pytest.mark.parametrize("form", ["decay", "sigmoid"])
def test_projection_recurrence_and_decode_together(form):
    """A gated recurrent layer as it is served and trained: int8 projection of the tokens to gate and
    input (the halves of one output, read in place), scan, int8 output projection; then the same layer token
    by token from the scan's state.  The projection's rows are independent of the batch they are in, so the
    decoded tokens see the same gates and inputs bit for bit, and the states differ only by the scan's
    order of composition."""
    batch, L, Dm, D = 2, 150, 256, 320
    r = torch.Generator().manual_seed(5)
    x = torch.randn(batch, L, Dm, generator=r).to(torch.bfloat16).cuda()
    w_in, w_out = int8(2 * D, Dm, 7), int8(Dm, D, 8)
    s_in = torch.full((2 * D,), 1 / (73 * Dm ** 0.5)).cuda()
    s_out = torch.full((Dm,), 1 / (73 * D ** 0.5)).cuda()
    b_in = torch.cat([torch.full((D,), 1.5 if form == "sigmoid" else -2.0), torch.zeros(D)]).cuda()

    def project(x):
        return jscan.matmul_i8(*jscan.quantize_rows(x), w_in, s_in, bias=b_in)

    def gates(p):   # the decay form's log gate has to be negative
        g, u = p[..., :D], p[..., D:]
        return (g if form == "sigmoid" else -torch.exp(g.float()).to(g.dtype)), u

    g, u = gates(project(x))
    y, h = jscan.gated_scan(g, u, form=form)
    out = jscan.matmul_i8(*jscan.quantize_rows(y), w_out, s_out)
    E, _ = O.scan_error(g, u, None, None, form)
    want_y, want_h = O.scan(g, u, None, None, form)
    assert (np.abs(f64(y) - want_y) <= E + 2.0 ** -8 * (np.abs(want_y) + E)).all()
    check_product(out.view(-1, Dm), *(t.view(-1, *t.shape[2:]) for t in jscan.quantize_rows(y)), w_out, s_out, None)

    _, s = jscan.gated_scan(*(v[:, :100] if v.stride(0) == 100 * v.stride(1) else v[:, :100].contiguous() for v in (g, u)),
                            form=form)
    for t in range(100, L):
        g_t, u_t = gates(project(x[:, t].contiguous()))
        assert torch.equal(bits(g_t), bits(g[:, t])) and torch.equal(bits(u_t), bits(u[:, t]))
        y_t = jscan.gated_step(s, g_t, u_t, form=form)
        assert (np.abs(f64(y_t) - want_y[:, t]) <= E[:, t] + 2.0 ** -8 * (np.abs(want_y[:, t]) + E[:, t])).all()
    assert (np.abs(f64(s) - want_h) <= E[:, -1] + 2.0 ** -24 * np.abs(want_h)).all()
    say(f"{form}: layer of {L} tokens, states within the bound")
    dy = torch.randn(batch, L, D, generator=r).to(torch.bfloat16).cuda()
    dproj = torch.empty(batch, L, 2 * D, dtype=torch.bfloat16, device="cuda")
    dg, du, dh0 = jscan.gated_scan_backward(g, u, y, dy, form=form, dg=dproj[..., :D], du=dproj[..., D:])
    Eg, Eu, E0 = O.backward_error(g, u, y, dy, None, None, None, form)
    dg_w, du_w, dh0_w, _ = O.backward(g, u, y, dy, None, None, None, form)
    for got, want, e in ((dproj[..., :D], dg_w, Eg), (dproj[..., D:], du_w, Eu)):
        assert (np.abs(f64(got) - want) <= e + 2.0 ** -8 * (np.abs(want) + e)).all()
    assert (np.abs(f64(dh0) - dh0_w) <= E0 + 2.0 ** -24 * np.abs(dh0_w)).all()

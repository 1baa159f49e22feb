"""The int8 product's epilogue on the GPU (activation, residual) against its definition in fp64, and a layer's calls in
a row.

Tolerance: the bound that the oracle derives (exact sum rounded once, two scale products, the bias sum, the
activation, the residual's sum) and half a step of the output's type."""
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


def product(M, N, K, seed=0):
    g = torch.Generator().manual_seed(M + N + K + seed)
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sq = torch.exp(0.5 * torch.randn(M, generator=g) - 4.5).cuda()
    sw = torch.exp(0.5 * torch.randn(N, generator=g) - 4.5).cuda() / K ** 0.5
    return q, sq, w, sw


def check(out, q, sq, w, sw, bias, act, residual, rows=slice(None)):
    want, err = O.matmul_i8(q[rows].cpu(), sq[rows], w.cpu(), sw, bias, act, None if residual is None else residual[rows])
    got = f64(out[rows])
    tol = err + torch.finfo(out.dtype).eps / 2 * (np.abs(want) + err) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{bad.sum()} of {bad.size} outside, first at {i}: {got[i]} against {want[i]} ({tol[i]})")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act,residual", [("silu", False), ("gelu_tanh", False), ("none", True), ("silu", True), ("gelu_tanh", True)])
@pytest.mark.parametrize("M,N,K", [   # every tile, with rows, columns and K that end inside one
    (1, 1, 16), (2, 17, 48), (16, 288, 128), (33, 64, 1040), (65, 127, 256), (100, 288, 8192), (129, 257, 272), (200, 1000, 64),
    (1, 4096, 8192), (77, 4096, 2064), (4, 5000, 2064), (1025, 65, 16), (256, 2100, 4112)])
def test_epilogue_matches_the_definition(M, N, K, act, residual, dtype):
    q, sq, w, sw = product(M, N, K)
    bias = normal(N, N).cuda() if M % 2 else None
    res = normal(M, M, N).to(DT[dtype]).cuda() if residual else None
    out = jscan.matmul_i8(q, sq, w, sw, bias=bias, out_dtype=DT[dtype], activation=act, residual=res)
    check(out, q, sq, w, sw, bias, act, res)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1000, 4100, 144), (2500, 2600, 1552), (6000, 6001, 96), (4096, 4090, 1040), (8200, 8301, 144),
                                   (20000, 288, 64), (190, 2050, 8208), (777, 2111, 2064), (512, 4100, 1040)])
def test_large_products(M, N, K, dtype):
    q, sq, w, sw = product(M, N, K)
    bias, res = normal(N, N).cuda(), normal(M, M, N).to(DT[dtype]).cuda()
    out = jscan.matmul_i8(q, sq, w, sw, bias=bias, out_dtype=DT[dtype], activation="silu", residual=res)
    v = ((q.double() @ w.double().t()) * sq.double()[:, None] * sw.double() + bias.double()).cpu().numpy()
    # the same bound as check(), with the exact integer sums formed on the GPU
    e = 4 * O.U * (np.abs(v) + np.abs(f64(bias)))
    want = O.activate(v, "silu") + f64(res)
    err = O.activate_error(v, e, "silu")
    err = err + O.U * (np.abs(want) + err)
    tol = err + torch.finfo(out.dtype).eps / 2 * (np.abs(want) + err) + 1e-37
    assert (np.abs(f64(out) - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,wide,start", [(64, 128, 64), (64, 65, 1), (100, 103, 3), (288, 576, 288), (7, 20, 13)])
def test_strided_residual_and_in_place(N, wide, start, dtype):
    M, K = 150, 208
    q, sq, w, sw = product(M, N, K)
    whole = normal(2, M, wide).to(DT[dtype]).cuda()
    before = whole.clone()
    stream = whole[:, start:start + N]
    want = jscan.matmul_i8(q, sq, w, sw, out_dtype=DT[dtype], activation="silu", residual=stream.contiguous())
    again = jscan.matmul_i8(q, sq, w, sw, out_dtype=DT[dtype], activation="silu", residual=stream)
    assert torch.equal(bits(again), bits(want))
    out = jscan.matmul_i8(q, sq, w, sw, out=stream, activation="silu", residual=stream)
    assert out is stream and torch.equal(bits(stream), bits(want))
    whole[:, start:start + N] = before[:, start:start + N]
    assert torch.equal(bits(whole), bits(before))


@pytest.mark.parametrize("M,N,K", [(3, 40, 96), (300, 520, 208)])
def test_no_epilogue_is_the_plain_call_and_special_rows(M, N, K):
    q, sq, w, sw = product(M, N, K)
    bias = normal(1, N).cuda()
    a = jscan.matmul_i8(q, sq, w, sw, bias=bias)
    b = jscan.matmul_i8(q, sq, w, sw, bias=bias, residual=torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(a, b)
    sq[1] = float("nan")   # a row that had no scale stays one, and alone
    res = normal(2, M, N).to(torch.bfloat16).cuda()
    res[2, 5] = float("inf")
    out = jscan.matmul_i8(q, sq, w, sw, bias=bias, activation="gelu_tanh", residual=res)
    assert torch.isnan(out[1]).all() and out[2, 5] == float("inf")
    keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
    keep[1], keep[2, 5] = False, False
    assert torch.isfinite(out[keep]).all()
    sq[1] = 1e30           # far ends of the activations
    for act in ("silu", "gelu_tanh"):
        out = jscan.matmul_i8(q, sq, w, sw, activation=act, out_dtype=torch.float32)
        v = (q[1].double() @ w.double().t()) * 1e30 * sw.double()
        assert torch.equal(out[1] > 0, v > 1e20) and (out[1][v < 0] == 0).all()


def layer(c, x, residual, conv_state, h, lengths=None):
    """One layer of the model as a serving program calls it: norm into 8 bits, projection to x and z, convolution,
    the scan's inputs, the scan with skip and gate, quantised projection into the residual stream."""
    q, s, total = jscan.rms_norm_quantize(x, c["gain"], residual=residual)
    xz = jscan.matmul_i8(q, s, c["w_in"], c["s_in"])
    D = c["skip"].shape[0]
    u, conv_state = jscan.causal_conv(xz[..., :D], c["taps"], bias=c["tap_bias"], state=conv_state, state_out=conv_state)
    delta, B, C, _ = jscan.ssm_inputs(u, c["w_x"], c["g_d"], c["g_B"], c["g_C"], c["w_dt"], c["b_dt"])
    y, h = jscan.prefill_gate(u, delta, c["A"], B, C, skip=c["skip"], z=xz[..., D:], h0=h, h_final=h)
    q, s = jscan.quantize_rows(y)
    return jscan.matmul_i8(q, s, c["w_out"], c["s_out"], residual=total), (u, delta, B, C, xz, y, total)


def weights(D, H, R):
    g = torch.Generator().manual_seed(5)
    i8 = lambda *s: (32 * torch.randn(*s, generator=g)).round().clamp(-127, 127).to(torch.int8).cuda()   # noqa: E731
    n = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    return dict(gain=1 + 0.2 * n(H), w_in=i8(2 * D, H), s_in=torch.full((2 * D,), 1 / (32 * H ** 0.5)).cuda(), taps=n(D, 4) / 2,
                tap_bias=0.2 * n(D), w_x=(n(R + 32, D) / D ** 0.5).to(torch.bfloat16), g_d=1 + 0.1 * n(R), g_B=1 + 0.1 * n(16),
                g_C=1 + 0.1 * n(16), w_dt=(n(D, R) / R ** 0.5).to(torch.bfloat16), b_dt=n(D) - 3,
                A=-torch.arange(1, 17).float().cuda().repeat(D, 1), skip=1 + 0.2 * n(D), w_out=i8(H, D),
                s_out=torch.full((H,), 1 / (32 * D ** 0.5)).cuda())


def test_a_layer_of_calls_prompt_then_tokens():
    """A prompt and the tokens behind it, each one through the single-token calls, against the whole sequence in one
    prompt: bit for bit where the calls promise it, and each call's inputs against the scan's oracle."""
    D, H, R, batch, L, more = 128, 96, 64, 2, 70, 5
    c = weights(D, H, R)
    x, res = (normal(i, batch, L + more, H).to(torch.bfloat16).cuda() for i in (1, 2))
    zeros = lambda: (torch.zeros(batch, 3, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(batch, D, 16, device="cuda"))   # noqa: E731
    conv_all, h_all = zeros()
    out_all, (u, delta, B, C, xz, y, total) = layer(c, x, res, conv_all, h_all)
    want = oracle.prefill(u, delta, c["A"], B, C)[0]
    want = (want + f64(c["skip"]) * f64(u)) * O.activate(f64(xz[..., D:]), "silu")
    assert_parity(f64(y), want, torch.bfloat16, "the scan with its gate inside the layer")

    conv, h = zeros()
    first, _ = layer(c, x[:, :L].contiguous(), res[:, :L].contiguous(), conv, h)
    assert torch.equal(bits(first), bits(out_all[:, :L]))
    for t in range(L, L + more):
        q, s, tot = jscan.rms_norm_quantize(x[:, t], c["gain"], residual=res[:, t])
        pair = jscan.matmul_i8(q, s, c["w_in"], c["s_in"])
        u_t = jscan.causal_conv_step(conv, pair[:, :D], c["taps"], bias=c["tap_bias"])
        d_t, B_t, C_t, _ = jscan.ssm_inputs(u_t, c["w_x"], c["g_d"], c["g_B"], c["g_C"], c["w_dt"], c["b_dt"])
        y_t = jscan.step_gate(h, u_t, d_t, c["A"], B_t, C_t, skip=c["skip"], z_t=pair[:, D:])
        q, s = jscan.quantize_rows(y_t)
        out = jscan.matmul_i8(q, s, c["w_out"], c["s_out"], residual=tot, out=tot)
        assert torch.equal(bits(u_t), bits(u[:, t])) and torch.equal(bits(pair), bits(xz[:, t]))
        assert_parity(f64(y_t), f64(y[:, t]), torch.bfloat16, f"y of token {t}")
        assert_parity(f64(out), f64(out_all[:, t]), torch.bfloat16, f"token {t}")
    assert torch.equal(bits(conv), bits(conv_all)) and torch.equal(bits(h), bits(h_all))


def test_a_training_step_of_norm_convolution_and_gated_scan():
    """The training calls in a row as an autograd function, against autograd through the formulas in fp64."""
    M, L, D = 2, 40, 48
    dev = lambda t: t.cuda()   # noqa: E731
    x, res, gain, taps, tb = (dev(normal(i, *s)) for i, s in enumerate([(M, L, D), (M, L, D), (D,), (D, 4), (D,)]))
    gate, dout = dev(normal(7, M, L, D)), dev(normal(8, M, L, D))
    n, total = jscan.rms_norm(x, gain, residual=res)
    u, _ = jscan.causal_conv(n, taps, bias=tb)
    y, _ = jscan.gated_scan(gate, u, form="sigmoid")
    dgate, du, _ = jscan.gated_scan_backward(gate, u, y, dout, form="sigmoid")
    dn, dtaps, dtb, _ = jscan.causal_conv_backward(n, taps, du, bias=tb)
    dx, dgain = jscan.rms_norm_backward(total, gain, dn, dtotal=dout)

    leaves = [t.double().cpu().requires_grad_() for t in (x, res, gain, taps, tb, gate)]
    X, Rz, G, T, Bz, S = leaves
    tot = X + Rz
    nn = tot * torch.rsqrt((tot ** 2).mean(-1, keepdim=True) + 1e-6) * G
    pad = torch.cat([torch.zeros(M, 3, D, dtype=torch.float64), nn], 1)
    v = Bz + sum(T[:, k] * pad[:, k:k + L] for k in range(4))
    uu, a, h, hs = v * torch.sigmoid(v), torch.sigmoid(S), torch.zeros(M, D, dtype=torch.float64), []
    for t in range(L):
        h = a[:, t] * h + (1 - a[:, t]) * uu[:, t]
        hs.append(h)
    out = torch.stack(hs, 1)
    ((out + tot) * dout.double().cpu()).sum().backward()
    for got, leaf, name in ((dx, X, "x"), (dx, Rz, "residual"), (dgain, G, "gain"), (dtaps, T, "taps"), (dtb, Bz, "bias"),
                            (dgate, S, "gate")):
        # a few hundred fp32 roundings deep, each 2^-24 of values of the size of the largest
        err = (got.double().cpu() - leaf.grad).abs().max() / leaf.grad.abs().max()
        assert err < 400 * 2.0 ** -24, (name, float(err))
    assert (y.double().cpu() - out).abs().max() < 400 * 2.0 ** -24 * out.abs().max()

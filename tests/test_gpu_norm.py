"""The root-mean-square norm on the GPU against its definition in fp64: with the residual's addition, into the tensor's
type and into 8 bits, and its gradients.

Tolerances: the bounds of the fp32 evaluation that the oracle derives, and half a step of the output's type
(torch.finfo(dtype).eps / 2 of the value)."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import bits, f64, say
from oracle import layer as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def same(a, b):
    return torch.equal(bits(a), bits(b))


def assert_within(got, want, err, what):
    tol = err + torch.finfo(got.dtype).eps / 2 * (np.abs(want) + err) + 1e-37
    g = f64(got)
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside, first at {i}: {g[i]} against {want[i]} ({tol[i]})")


# one piece a thread and more, one, four and sixteen waves, pieces that end inside a row, rows element by element
SHAPES = [(1, 1), (3, 2), (2, 3), (5, 4), (4, 7), (3, 8), (2, 9), (7, 16), (3, 100), (2, 511), (9, 512), (1, 513), (4, 1000),
          (2, 1024), (3, 1025), (2, 2049), (5, 4096), (1, 4100), (2, 8191), (2, 8200), (1, 16384), (2, 20001), (1, 32768),
          (2, 32769), (1, 50001), (300, 64), (9000, 24), (3000, 300)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_norm_matches_the_definition(M, K, dtype):
    x, res, gain = normal(M, M, K).to(DT[dtype]), normal(K, M, K).to(DT[dtype]), 1 + 0.3 * normal(3, K)
    y, total = jscan.rms_norm(x.cuda(), gain.cuda(), residual=res.cuda())
    assert same(total, (x.float() + res.float()).to(DT[dtype]))
    assert_within(y, *O.rms_norm(total, gain, 1e-6), "y")
    alone, back = jscan.rms_norm(total, gain.cuda())
    assert back is total and same(alone, y)
    y, total = jscan.rms_norm(x.cuda(), gain.cuda(), eps=0.5)
    assert_within(y, *O.rms_norm(x, gain, 0.5), "y alone")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (5, 80), (1, 4096), (33, 4112), (7, 8192), (300, 1024), (2, 131056), (1030, 256),
                                 (2, 16400), (4, 32784), (9000, 32)])
def test_eight_bit_output(M, K, dtype):
    """Scales to their rounding; quantised values that stand for y to half a quantum and y's own error."""
    x, res = (normal(M, M, K) * torch.exp(2 * normal(1, M, 1))).to(DT[dtype]), normal(K, M, K).to(DT[dtype])
    gain = 1 + 0.3 * normal(3, K)
    q, scale, total = jscan.rms_norm_quantize(x.cuda(), gain.cuda(), residual=res.cuda())
    assert q.shape == (M, K) and scale.shape == (M,) and same(total, (x.float() + res.float()).to(DT[dtype]))
    y, err = O.rms_norm(total, gain, 1e-6)
    s = f64(scale)
    want = np.abs(y).max(1) / 127
    assert (np.abs(s - want) <= err.max(1) / 127 + 2 * 2.0 ** -24 * want).all()
    # rint of y (1 / s): the reciprocal and the product round once each
    off = np.abs(f64(q) * s[:, None] - y)
    assert (off <= 0.5 * s[:, None] + err + 2 * 2.0 ** -24 * np.abs(y)).all()
    q2, scale2, _ = jscan.rms_norm_quantize(total, gain.cuda())
    assert torch.equal(q, q2) and same(scale, scale2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_gradients_match_the_definition(M, K, dtype):
    total, dy, gain = normal(M, M, K).to(DT[dtype]), normal(K + 1, M, K).to(DT[dtype]), 1 + 0.3 * normal(3, K)
    dtotal = normal(9, M, K).to(DT[dtype]) if K % 2 else None
    dx, dgain = jscan.rms_norm_backward(total.cuda(), gain.cuda(), dy.cuda(), dtotal=None if dtotal is None else dtotal.cuda())
    want, want_gain, e, e_gain = O.rms_norm_backward(total, gain, dy, dtotal, 1e-6)
    assert_within(dx, want, e, "dx")
    assert_within(dgain, want_gain, e_gain, "dgain")


def test_gradients_against_differences():
    M, K, eps = 5, 96, 0.1
    x, res, gain = (normal(i, M, K).cuda() for i in (1, 2, 3))
    gain, dy, dt = 1 + 0.3 * gain[0], normal(4, M, K).cuda(), normal(5, M, K).cuda()

    def loss(x, res, gain):
        y, total = jscan.rms_norm(x.contiguous(), gain, residual=res, eps=eps)
        return float((y.double() * dy.double()).sum() + (total.double() * dt.double()).sum())

    _, total = jscan.rms_norm(x, gain, residual=res, eps=eps)
    dx, dgain = jscan.rms_norm_backward(total, gain, dy, dtotal=dt, eps=eps)
    h = 2.0 ** -8
    for name, g, at in (("x", dx, 0), ("residual", dx, 1), ("gain", dgain, 2)):
        up, down = [x, res, gain], [x, res, gain]
        up[at], down[at] = up[at] + h * g.sign(), down[at] - h * g.sign()
        slope, want = (loss(*up) - loss(*down)) / (2 * h), float(g.double().abs().sum())
        # a step of h per element moves a row of rms 1.4 by at most h relative to it, and the norm's third derivative
        # along such a step is below 16 / rms^3: h^2 / 6 * 16 < 5e-5 of the sum of |dy|; fp32 adds 2^-23 / h of it
        say(f"d{name}: {slope:.6g} by differences, {want:.6g}")
        assert abs(slope - want) <= 1e-4 * float(dy.double().abs().sum())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,wide,start", [(64, 128, 64), (64, 65, 1), (48, 71, 5), (4096, 4099, 3), (7, 20, 13), (112, 112, 0)])
def test_strided_rows_and_leading_dimensions(K, wide, start, dtype):
    def cut(t):
        return t[..., start:start + K]

    gain = (1 + 0.3 * normal(3, K)).cuda()
    x, res, dy = (normal(i, 3, 5, wide).to(DT[dtype]).cuda() for i in (1, 2, 4))
    whole, sums = (torch.full((3, 5, wide), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    y, total = jscan.rms_norm(cut(x), gain, residual=cut(res), y=cut(whole), total=cut(sums))
    y0, total0 = jscan.rms_norm(cut(x).contiguous(), gain, residual=cut(res).contiguous())
    assert same(y, y0) and same(total, total0) and y0.shape == (3, 5, K)
    cut(whole).fill_(7)
    dx, dgain = jscan.rms_norm_backward(total, gain, cut(dy), dtotal=cut(x), dx=cut(whole))
    dx0, dgain0 = jscan.rms_norm_backward(total0, gain, cut(dy).contiguous(), dtotal=cut(x).contiguous())
    assert same(dx, dx0) and same(dgain, dgain0)
    cut(whole).fill_(7)
    cut(sums).fill_(7)
    assert (whole == 7).all() and (sums == 7).all()
    if K % 16 == 0:
        q, s, _ = jscan.rms_norm_quantize(cut(x), gain, residual=cut(res))
        q0, s0, _ = jscan.rms_norm_quantize(cut(x).contiguous(), gain, residual=cut(res).contiguous())
        assert torch.equal(q, q0) and same(s, s0) and q.shape == (3, 5, K) and s.shape == (3, 5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 100, 1021, 4096, 8197, 20001, 40001])
def test_in_place(K, dtype):
    """The residual stream updated in place, and a gradient added into."""
    M = 37
    gain = (1 + 0.3 * normal(3, K)).cuda()
    x, res, dy = (normal(i, M, K).to(DT[dtype]).cuda() for i in (1, 2, 4))
    y, total = jscan.rms_norm(x, gain, residual=res)
    for into in ("x", "residual"):
        a = {"x": x.clone(), "residual": res.clone()}
        y2, t2 = jscan.rms_norm(a["x"], gain, residual=a["residual"], total=a[into])
        assert t2 is a[into] and same(t2, total) and same(y2, y)
    dx, dgain = jscan.rms_norm_backward(total, gain, dy, dtotal=x)
    d = x.clone()
    dx2, dgain2 = jscan.rms_norm_backward(total, gain, dy, dtotal=d, dx=d)
    assert dx2 is d and same(d, dx) and same(dgain, dgain2)


@pytest.mark.parametrize("K", [16385, 16391, 16897, 24577, 24583])
def test_gradient_added_into_where_long_rows_are_read_again(K):
    """The last piece of such a row reaches back over elements that other threads have written already."""
    M = 600
    gain = (1 + 0.3 * normal(3, K)).cuda()
    total, dy, dtotal = (normal(i, M, K).to(torch.bfloat16).cuda() for i in (1, 2, 4))
    dx, dgain = jscan.rms_norm_backward(total, gain, dy, dtotal=dtotal)
    for _ in range(3):
        d = dtotal.clone()
        dx2, dgain2 = jscan.rms_norm_backward(total, gain, dy, dtotal=d, dx=d)
        assert dx2 is d and same(d, dx) and same(dgain, dgain2)


@pytest.mark.parametrize("K", [48, 4096, 65536])
def test_special_rows(K):
    M = 8
    x = normal(1, M, K).cuda()
    gain = (1 + 0.3 * normal(3, K)).cuda()
    x[0], x[1, K - 1], x[2, 0], x[3, K // 2], x[4] = 0, float("nan"), float("inf"), -float("inf"), 1e-25
    x[5] = 1e30   # the squares overflow
    y, _ = jscan.rms_norm(x, gain)
    q, s, _ = jscan.rms_norm_quantize(x, gain)
    assert not y[0].any() and not q[0].any() and torch.isfinite(s[0])
    assert torch.isnan(y[1]).all() and torch.isnan(s[1:4]).all() and torch.isnan(s[5]) and not q[1:4].any()
    for ok in (0, 4, 6, 7):
        assert torch.isfinite(y[ok]).all()
        assert_within(y[ok], *O.rms_norm(x[ok], gain, 1e-6), f"row {ok}")
    bad = gain.clone()
    bad[3] = float("nan")
    _, s, _ = jscan.rms_norm_quantize(x[6:], bad)
    assert torch.isnan(s).all()


def test_no_rows_and_one_dimension():
    gain = torch.ones(32, device="cuda")
    y, total = jscan.rms_norm(torch.empty(0, 32, device="cuda"), gain, residual=torch.empty(0, 32, device="cuda"))
    assert y.shape == total.shape == (0, 32)
    q, s, _ = jscan.rms_norm_quantize(torch.empty(4, 0, 32, device="cuda"), gain)
    assert q.shape == (4, 0, 32) and s.shape == (4, 0)
    dx, dgain = jscan.rms_norm_backward(torch.empty(0, 32, device="cuda"), gain, torch.empty(0, 32, device="cuda"),
                                        dgain=torch.full((32,), 3.0, device="cuda"))
    assert dx.shape == (0, 32) and not dgain.any()
    x = normal(1, 32).cuda()
    y, _ = jscan.rms_norm(x, gain)
    q, s, _ = jscan.rms_norm_quantize(x, gain)
    assert y.shape == (32,) and q.shape == (32,) and s.shape == ()
    assert_within(y[None], *O.rms_norm(x[None], gain, 1e-6), "one row")


def test_captured_and_replayed_and_on_another_stream():
    M, K = 700, 520
    gain = (1 + 0.3 * normal(3, K)).cuda()
    x, res, dy = (normal(i, M, K).to(torch.bfloat16).cuda() for i in (1, 2, 4))
    ws = torch.empty(jscan.rms_norm_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")

    def work():
        y, total = jscan.rms_norm(x, gain, residual=res)
        dx, dgain = jscan.rms_norm_backward(total, gain, dy, dtotal=res, workspace=ws)
        q, s, _ = jscan.rms_norm_quantize(x[:, :512], gain[:512], residual=res[:, :512])
        return [y, total, dx, dgain, q, s]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        x.copy_(normal(20 + i, M, K))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = work()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {i}"

"""Refusals of the gated recurrence's and the int8 projection's entry points, before any launch (the
addresses below are never dereferenced), and of their binding.  CPU only."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EALIAS, EHIP, EWORKSPACE, EFORM = range(9)
F32, BF16 = 0, 1
P = 0x100000000
STEP = 0x10000000


def scan(**kw):
    a = dict(g=P, u=P + STEP, h0=None, n=None, y=P + 2 * STEP, h=P + 3 * STEP, batch=2, L=64, D=64, ld_g=64, ld_u=64,
             ld_y=64, ws=P + 8 * STEP, ws_bytes=1 << 40, form=0, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_gated_scan(*a.values(), None)


def backward(**kw):
    a = dict(g=P, u=P + STEP, y=P + 2 * STEP, dy=P + 3 * STEP, h0=None, dh=None, n=None, dg=P + 4 * STEP,
             du=P + 5 * STEP, dh0=None, batch=2, L=64, D=64, ld_g=64, ld_u=64, ld_y=64, ld_dy=64, ld_dg=64, ld_du=64,
             ws=P + 8 * STEP, ws_bytes=1 << 40, form=1, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_gated_scan_backward(*a.values(), None)


def step(**kw):
    a = dict(h=P, g=P + STEP, u=P + 2 * STEP, y=P + 3 * STEP, batch=2, D=64, ld_g=64, ld_u=64, ld_y=64, form=0,
             dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_gated_step(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(form=2), EFORM), (dict(form=-1), EFORM), (dict(dtype=7), EDTYPE), (dict(batch=-1), ESHAPE),
    (dict(L=-1), ESHAPE), (dict(D=-8), ESHAPE), (dict(D=(1 << 24) + 1), ESHAPE), (dict(batch=(1 << 20) + 1), ESHAPE),
    (dict(L=1 << 31), ESHAPE), (dict(ld_g=63), ESHAPE), (dict(ld_u=0), ESHAPE), (dict(ld_y=-64), ESHAPE),
    (dict(ld_g=1 << 58), ESHAPE), (dict(g=None), ENULL), (dict(u=None), ENULL), (dict(y=None), ENULL),
    (dict(h=None), ENULL), (dict(g=P + 1), EALIGN), (dict(y=P + 2 * STEP + 1), EALIGN), (dict(dtype=F32, u=P + 2), EALIGN),
    (dict(h=P + 3 * STEP + 2), EALIGN), (dict(n=P + 7 * STEP + 1), EALIGN), (dict(y=P), EALIAS), (dict(y=P + STEP + 128), EALIAS),
    (dict(h=P + STEP), EALIAS), (dict(h0=P + 3 * STEP + 4), EALIAS), (dict(n=P + 2 * STEP), EALIAS),
    # the halves of one buffer are apart, columns that cross are not
    (dict(y=P + 100, ld_g=128, ld_u=128, ld_y=128), EALIAS), (dict(y=P + 128, ld_g=128, ld_y=130), EALIAS),
    (dict(batch=0, g=None, u=None, y=None, h=None), OK), (dict(D=0, h=None), OK),
])
def test_scan_validation(kw, code):
    assert scan(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(form=9), EFORM), (dict(dtype=2), EDTYPE), (dict(L=-3), ESHAPE), (dict(ld_dg=60), ESHAPE),
    (dict(ld_u=1), ESHAPE), (dict(u=None), ENULL), (dict(y=None), ENULL), (dict(dy=None), ENULL),
    (dict(dg=None), ENULL), (dict(du=None), ENULL), (dict(dg=P + 4 * STEP + 1), EALIGN), (dict(dh0=P + 6 * STEP + 2), EALIGN),
    (dict(dg=P), EALIAS), (dict(du=P + 3 * STEP), EALIAS), (dict(du=P + 4 * STEP), EALIAS),
    (dict(dh0=P + 6 * STEP, dh=P + 6 * STEP + 256), EALIAS), (dict(dh0=P + 4 * STEP), EALIAS),
    (dict(h0=P + 6 * STEP, dh0=P + 6 * STEP), EALIAS),
    (dict(dg=P + 4 * STEP, du=P + 4 * STEP + 64, ld_dg=128, ld_du=128), EALIAS),
    (dict(batch=0), OK), (dict(D=0), OK),
])
def test_backward_validation(kw, code):
    assert backward(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(form=3), EFORM), (dict(dtype=5), EDTYPE), (dict(batch=-1), ESHAPE), (dict(ld_y=10), ESHAPE),
    (dict(h=None), ENULL), (dict(g=None), ENULL), (dict(h=P + 2), EALIGN), (dict(u=P + 2 * STEP + 1), EALIGN),
    (dict(y=P), EALIAS), (dict(y=P + STEP), EALIAS), (dict(h=P + STEP), EALIAS), (dict(batch=0, h=None), OK),
])
def test_step_validation(kw, code):
    assert step(**kw) == code


def quantize(**kw):
    a = dict(x=P, q=P + STEP, s=P + 2 * STEP, M=8, K=64, ld=64, dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_quantize_rows(*a.values(), None)


def matmul(**kw):
    a = dict(q=P, sq=P + STEP, w=P + 2 * STEP, sw=P + 3 * STEP, bias=None, out=P + 4 * STEP, M=8, N=24, K=64, ld=24,
             dtype=BF16)
    a.update(kw)
    return jscan.library().jscan_matmul_i8(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), EDTYPE), (dict(M=-1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=72, ld=72), ESHAPE), (dict(ld=63), ESHAPE),
    (dict(K=131072, ld=131072), ESHAPE), (dict(x=None), ENULL), (dict(q=None), ENULL), (dict(s=None), ENULL),
    (dict(x=P + 1), EALIGN), (dict(q=P + STEP + 8), EALIGN), (dict(s=P + 2 * STEP + 2), EALIGN), (dict(q=P), EALIAS),
    (dict(s=P + STEP), EALIAS), (dict(s=P + 16), EALIAS), (dict(M=0, x=None), OK),
])
def test_quantize_validation(kw, code):
    assert quantize(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), EDTYPE), (dict(M=-1), ESHAPE), (dict(N=-1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=24), ESHAPE),
    (dict(K=131072), ESHAPE), (dict(ld=23), ESHAPE), (dict(M=1 << 30, N=1 << 24, ld=1 << 24), ESHAPE),
    (dict(q=None), ENULL), (dict(sq=None), ENULL), (dict(w=None), ENULL), (dict(sw=None), ENULL), (dict(out=None), ENULL),
    (dict(q=P + 8), EALIGN), (dict(w=P + 2 * STEP + 4), EALIGN), (dict(out=P + 4 * STEP + 1), EALIGN),
    (dict(bias=P + 5 * STEP + 1), EALIGN), (dict(out=P), EALIAS), (dict(out=P + 3 * STEP), EALIAS),
    (dict(bias=P + 4 * STEP), EALIAS), (dict(M=0), OK), (dict(N=0), OK),
])
def test_matmul_validation(kw, code):
    assert matmul(**kw) == code


def test_workspace_sizes():
    lib = jscan.library()
    assert lib.jscan_gated_scan_workspace(0, 10, 10) == 0 and lib.jscan_gated_scan_workspace(4, 0, 64) == 0
    assert lib.jscan_gated_scan_workspace(-1, 10, 10) == -1 and lib.jscan_gated_scan_workspace(1, 1 << 31, 8) == -1
    for batch, L, D in ((1, 65536, 1024), (16, 4096, 8192), (3, 77, 1000), (1, 1, 1), (1 << 20, 1, 1 << 10)):
        n = lib.jscan_gated_scan_workspace(batch, L, D)
        assert 0 <= n <= batch * L * D * 4
        assert jscan.gated_scan_workspace_bytes(batch, L, D) == n
        if n > 0:   # a missing, short or misaligned workspace is refused
            far = dict(u=P + 64 * STEP, y=P + 128 * STEP, h=P + 192 * STEP, ws=P + 256 * STEP, batch=batch, L=L, D=D,
                       ld_g=D, ld_u=D, ld_y=D)
            assert scan(**{**far, "ws": None}) == ENULL
            assert scan(**far, ws_bytes=n - 1) == EWORKSPACE
            assert scan(**{**far, "ws": P + 256 * STEP + 4}) == EALIGN
            assert scan(**{**far, "ws": P + 64 * STEP}) == EALIAS
    with pytest.raises(ValueError):
        jscan.gated_scan_workspace_bytes(1, -1, 8)


def test_binding_refuses_before_the_library():
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        jscan.gated_scan(x, x)
    with pytest.raises(ValueError, match="form"):
        jscan.gated_scan(x, x, form="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        jscan.gated_scan_backward(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        jscan.gated_step(torch.zeros(2, 8), x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        jscan.quantize_rows(x)
    with pytest.raises(ValueError, match="CUDA"):
        jscan.matmul_i8(torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2), torch.zeros(4, 16, dtype=torch.int8),
                        torch.zeros(4))


def test_workspaces_that_are_not_memory_of_their_size_are_refused():
    from mamba_selective_scan_03_amd._binding import _gated_workspace

    need = jscan.gated_scan_workspace_bytes(1, 65536, 64)
    assert need > 0
    dev = torch.device("cpu")
    ws = torch.empty(need, dtype=torch.uint8)
    assert _gated_workspace(ws, 1, 65536, 64, dev) == (ws, need)
    assert _gated_workspace(torch.empty(3, dtype=torch.float64), 1, 65536, 64, dev)[1] == 24   # the library refuses it
    for bad in (torch.empty(1, dtype=torch.uint8).expand(need), torch.empty(2 * need, dtype=torch.uint8)[::2],
                torch.empty(need, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            _gated_workspace(bad, 1, 65536, 64, dev)


def test_token_rows_of_views():
    from mamba_selective_scan_03_amd._binding import _token_rows

    like = torch.zeros(1)
    wide = torch.zeros(3, 5, 24)
    assert _token_rows("t", wide, like, wide.shape) == 24
    assert _token_rows("t", wide[..., 8:16], like, (3, 5, 8)) == 24
    assert _token_rows("t", wide[:, :1, :8], like, (3, 1, 8)) == 120
    assert _token_rows("t", wide[1:2, 2:4, :8], like, (1, 2, 8)) == 24
    for bad, shape in ((wide[:, :4], (3, 4, 24)), (wide.transpose(1, 2), (3, 24, 5)), (wide[..., ::2], (3, 5, 12)),
                       (wide.double(), wide.shape), (wide, (3, 5, 8))):
        with pytest.raises(ValueError):
            _token_rows("t", bad, like, torch.Size(shape))


def test_row_strides_of_views():
    from mamba_selective_scan_03_amd._binding import _row_stride

    wide = torch.zeros(3, 5, 24)
    assert _row_stride("t", wide) == 24 and _row_stride("t", wide[..., :16]) == 24 and _row_stride("t", wide[0, 0]) == 24
    assert _row_stride("t", wide[:, :1, :16]) == 120 and _row_stride("t", wide[:1, 1:3, 8:]) == 24
    assert _row_stride("t", wide[0, 0, :16]) == 16 and _row_stride("t", wide[:0]) == 24
    for bad in (wide[:, :4], wide[..., ::2], wide.transpose(0, 1)):
        with pytest.raises(ValueError):
            _row_stride("t", bad)

"""The norm's backward pass over a few rows: a short pass in one launch, longer ones over work-groups of their own, which
leave their shares of the gain's gradient in the workspace and touch nothing behind it."""
import numpy as np
import pytest
import torch

import mamba_selective_scan_03_amd as jscan
from gpu_util import f64
from oracle import layer as O

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def test_long_rows_are_dealt_out():
    """A work-group walks its rows one after the other, so only a small pass is left to one (which needs no workspace)."""
    size = jscan.rms_norm_workspace_bytes
    for M, K in ((8, 4096), (2, 65536), (3, 16384), (8, 16384), (5, 1 << 20), (8, 1 << 24)):
        assert size(M, K) >= 2 * 4 * K
    for M, K in ((1, 64), (1, 16384), (1, 1 << 24), (8, 64), (8, 2048), (4, 4096), (2, 8192), (0, 4096)):
        assert size(M, K) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [7, 1000, 3001, 4096, 9000, 16384, 16400, 40000])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8])
def test_gradients_match_the_definition(M, K, dtype):
    gen = torch.Generator().manual_seed(M * K)
    total, dy, dtotal = (torch.randn(M, K, generator=gen).to(DT[dtype]) for _ in range(3))
    gain = 1 + 0.3 * torch.randn(K, generator=gen)
    n = jscan.rms_norm_workspace_bytes(M, K)
    room = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    dx, dgain = jscan.rms_norm_backward(total.cuda(), gain.cuda(), dy.cuda(), dtotal=dtotal.cuda(), workspace=room[:n])
    assert (room[n:] == 77).all()
    want, want_gain, e, e_gain = O.rms_norm_backward(total, gain, dy, dtotal, 1e-6)
    for got, ref, err in ((dx, want, e), (dgain, want_gain, e_gain)):
        assert (np.abs(f64(got) - ref) <= err + torch.finfo(got.dtype).eps / 2 * (np.abs(ref) + err) + 1e-37).all()

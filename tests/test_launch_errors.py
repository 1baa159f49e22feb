"""A launch that HIP refuses comes back as an error status from every entry point, whichever source file it is in: here
there is no GPU, so every launch is refused (the addresses are never dereferenced).  CPU only."""
import pytest
import torch

import mamba_selective_scan_03_amd as jscan

EHIP = 6
P, S = 0x100000000, 0x10000000
A = [P + i * S for i in range(16)]

CALLS = {
    "jscan_prefill": [*A[:7], 2, 8, 64, 16, 1],
    "jscan_step": [*A[:7], 2, 64, 16, 64, 16, 64, 1],
    "jscan_prefill_gate": [*A[:5], None, *A[5:9], 2, 8, 64, 16, 64, -1, None, 0, 0, 1],
    "jscan_step_gate": [*A[:9], 2, 64, 16, 64, 16, 64, 64, 0, 1],
    "jscan_gated_scan": [A[0], A[1], None, None, A[2], A[3], 2, 8, 64, 64, 64, 64, None, 0, 0, 1],
    "jscan_gated_step": [*A[:4], 2, 64, 64, 64, 64, 0, 1],
    "jscan_quantize_rows": [*A[:3], 8, 64, 64, 1],
    "jscan_matmul_i8": [*A[:4], None, A[4], 8, 64, 64, 64, 1],
    "jscan_matmul_i8_epilogue": [*A[:4], None, A[5], A[4], 8, 64, 64, 64, 64, 1, 1],
    "jscan_causal_conv": [A[0], None, A[1], None, None, A[2], A[3], 2, 8, 64, 4, 64, 64, 1, 1],
    "jscan_causal_conv_backward": [A[0], None, A[1], None, None, A[2], None, A[3], None, A[4], None, 2, 8, 64, 4, 64, 64, 64, A[5],
                                   1 << 20, 1, 1],
    "jscan_causal_conv_step": [*A[:3], None, A[3], 2, 64, 4, 64, 64, 1, 1],
    "jscan_rms_norm": [A[0], A[1], A[2], A[3], A[4], 8, 64, 64, 64, 64, 64, 1e-6, 1],
    "jscan_rms_norm_quantize": [*A[:6], 8, 64, 64, 64, 64, 1e-6, 1],
    "jscan_rms_norm_backward": [*A[:6], 8, 64, 64, 64, 64, 64, A[6], 1 << 20, 1e-6, 1],
}


@pytest.mark.skipif(torch.cuda.is_available(), reason="launches would run")
@pytest.mark.parametrize("name", CALLS)
def test_refused_launches_are_errors(name):
    lib = jscan.library()
    assert getattr(lib, name)(*CALLS[name], None) == EHIP
    assert lib.jscan_last_hip_error() != 0

"""The oracle's bound on the gradient of the norm's gain is narrow enough to miss no row: leaving out any one of the
rows of the largest shape that the GPU tests compare moves some column by more than the bound.  CPU only."""
import numpy as np
import pytest
import torch

from oracle import layer as O


@pytest.mark.parametrize("M,K", [(9000, 24), (3000, 300), (300, 64)])
def test_a_missing_row_exceeds_the_bound(M, K):
    gen = torch.Generator().manual_seed(M + K)
    total, dy = torch.randn(M, K, generator=gen), torch.randn(M, K, generator=gen)
    gain = 1 + 0.3 * torch.randn(K, generator=gen)
    _, dgain, _, e_gain = O.rms_norm_backward(total, gain, dy, None, 1e-6)
    t = total.double().numpy()
    terms = dy.double().numpy() * t / np.sqrt((t * t).mean(1, keepdims=True) + 1e-6)
    assert np.allclose(terms.sum(0), dgain, rtol=1e-12, atol=1e-12)
    tol = e_gain + 2.0 ** -24 * (np.abs(dgain) + e_gain)   # the gradient is fp32
    assert (np.abs(terms) > tol).any(1).all()

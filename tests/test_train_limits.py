"""Limits of the training calls' arguments, on the host (fake addresses, only where no GPU is visible)."""
import pytest
import torch

from test_train_abi import NO_DEVICE, embed, embed_backward, embed_f32, pre

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses: only where no GPU is visible")


@pytest.mark.parametrize("n", [1, 4, 8])
def test_iterations_that_the_history_cannot_index(n):
    assert pre(n=n, iters=2 ** 21 - 1) == NO_DEVICE
    for B in (0, 1, 4):
        assert pre(n=n, B=B, iters=2 ** 21) == mhc.MHC_ERR_UNSUPPORTED
        assert pre(n=n, B=B, iters=2 ** 31 - 1) == mhc.MHC_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [embed, embed_f32, embed_backward])
def test_every_finite_scale_is_taken(call):
    largest = 3.4028234663852886e38
    for scale in (largest, -largest, 3.1e38, 2.0 ** -149, 0.0):
        assert call(scale=scale) == NO_DEVICE, scale
    assert call(scale=3.5e38) == mhc.MHC_ERR_INVALID  # infinite in fp32

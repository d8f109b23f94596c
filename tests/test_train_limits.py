"""Limits of the training calls' arguments, on the host (fake addresses, only where no GPU is visible)."""
import pytest
import torch

from test_train_abi import NO_DEVICE, pre

mhc = pytest.importorskip("gemm_rms_sinkhorn_gb300")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses: only where no GPU is visible")


@pytest.mark.parametrize("n", [1, 4, 8])
def test_iterations_that_the_history_cannot_index(n):
    assert pre(n=n, iters=2 ** 21 - 1) == NO_DEVICE
    for B in (0, 1, 4):
        assert pre(n=n, B=B, iters=2 ** 21) == mhc.MHC_ERR_UNSUPPORTED
        assert pre(n=n, B=B, iters=2 ** 31 - 1) == mhc.MHC_ERR_UNSUPPORTED

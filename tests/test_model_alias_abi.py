"""Inputs of the norms that are one buffer, and outputs in their place: what the host's checks let through
(fake addresses, as in test_model_abi.py)."""
import pytest
import torch

from test_model_abi import NO_DEVICE, P, add, add_q8, back, mhc

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses: only where no GPU is visible")


@pytest.mark.parametrize("call", [add, add_q8])
def test_a_sum_of_one_buffer_with_itself(call):
    assert call(R=P[0]) == NO_DEVICE  # A + A
    assert call(R=P[0], H=P[0]) == NO_DEVICE  # and in its place
    assert call(R=P[0], H=P[0] + 16) == mhc.MHC_ERR_INVALID


def test_a_gradient_that_is_both_of_the_backwards():
    assert back(skip=P[0]) == NO_DEVICE
    assert back(skip=P[0], dH=P[0]) == NO_DEVICE
    assert back(H=P[0], dH=P[0]) == NO_DEVICE  # H is dZ, too
    assert back(dH=P[1]) == mhc.MHC_ERR_INVALID  # H alone may not be

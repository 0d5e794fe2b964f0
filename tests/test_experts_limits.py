"""The largest sizes of the expert-row calls (host only: the checks run before any
CUDA call, so a well-formed call answers "no device" here)."""
import pytest
import torch

from test_experts_abi import NO_DEVICE, UNSUPPORTED, combine, combine_grad, gather

HAS_GPU = torch.cuda.is_available()
MOST = 1 << 30  # choices of a token: combine and its gradient count past them in 32 bits


@pytest.mark.parametrize("call", [combine, combine_grad])
@pytest.mark.parametrize("s", [MOST + 1, (1 << 31) - 8, (1 << 31) - 1])
def test_choices_that_32_bits_cannot_step_through(call, s):
    assert call(T=1, S=s) == UNSUPPORTED
    assert call(T=0, S=s) == UNSUPPORTED


@pytest.mark.skipif(HAS_GPU, reason="would launch on stand-in pointers")
def test_choices_within_the_limit():
    assert combine(T=1, S=MOST) == NO_DEVICE and combine_grad(T=1, S=MOST) == NO_DEVICE
    assert gather(T=1, S=(1 << 31) - 1) == NO_DEVICE  # (walks in unsigned 32 bits)

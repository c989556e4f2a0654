"""Ends of the range of the routed sum's gradient."""
import pytest
import torch

from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_more_tokens_than_one_launch_takes():
    """2^26 tokens of eight columns and a few are more than 2^24 blocks of 256 threads; a grid
    holds fewer than 2^32 threads.  The last tokens are computed like the first."""
    T, H = (1 << 26) + 5, 8
    dout = torch.empty(T, H, dtype=BF, device="cuda").fill_(0.5)
    y = torch.empty(T, H, dtype=BF, device="cuda").fill_(2.0)
    last = torch.arange(1, 8, device="cuda").to(BF)
    dout[-7:], y[-7:] = last.unsqueeze(1), 3.0
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(T, 1, dtype=F32, device="cuda")
    r = ops.combine_backward(dout, y, ids, w, 1)
    assert torch.equal(r["dy"], dout)
    assert torch.equal(r["dw"][-7:, 0], 24 * last.float())
    assert bool((r["dw"][:-7] == 8.0).all())
    assert not bool(r["dlogits"].any())

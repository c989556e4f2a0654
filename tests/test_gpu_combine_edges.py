"""Ends of the range of the routed sum's gradient."""
import pytest
import torch

import _block_ref as R
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


@pytest.mark.parametrize("H", [64, 1032])
def test_a_dropped_pairs_weight_counts_nothing(H):
    """A pair whose id no expert has takes no part in the token's sums, whatever its
    weight is."""
    T, E, k = 9, 5, 3
    g = torch.Generator("cuda")
    g.manual_seed(H)
    z = torch.randn(T, E, generator=g, device="cuda")
    ids, w = ops.route(z, k)
    y, dout = (torch.randn(n, H, generator=g, device="cuda") for n in (T * k, T))
    ids[2, 1], ids[4, 0], ids[8, 2] = E, -7, 1 << 30
    w[2, 1], w[4, 0], w[8, 2] = float("nan"), float("inf"), 7.0
    gone = (ids < 0) | (ids >= E)
    wd = torch.where(gone, torch.zeros_like(w), w).double()
    terms = (dout.double().unsqueeze(1) * y.double().view(T, k, H)) * ~gone.unsqueeze(2)
    dw, mag = terms.sum(2), terms.abs().sum(2)
    mean = (wd * dw).sum(1, keepdim=True)
    dz = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    dz.scatter_add_(1, ids.long().clamp(0, E - 1), wd * (dw - mean) * ~gone)
    # a lane's chain of H / 64 products, a tree over the lanes and waves; then k products
    edw = (H / 64 + 12) * R.U32 * mag
    spread = wd * (edw + (wd * edw).sum(1, keepdim=True)
                   + (k + 4) * R.U32 * (dw.abs() + (wd * dw.abs()).sum(1, keepdim=True)))
    r = ops.combine_backward(dout, y, ids, w, E)
    assert not r["dy"].view(T, k, H)[gone].any() and not r["dw"][gone].any()
    assert ((r["dw"].double() - dw).abs() <= edw).all()
    edz = torch.zeros_like(dz).scatter_add_(1, ids.long().clamp(0, E - 1), spread * ~gone)
    assert ((r["dlogits"].double() - dz).abs() <= edz * 1.01 + 2 * R.U32 * dz.abs()).all()

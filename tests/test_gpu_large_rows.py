"""Routing, the weighted sum and the norms of more rows than one axis of a grid takes:
a grid with 2^32 threads or more along an axis runs, without an error, only what is left
of them behind 32 bits."""
import pytest
import torch

from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_route():
    """2^26 tokens and a few, four to a block of 256 threads."""
    T = (1 << 26) + 3
    z = torch.zeros(T, 2, dtype=F32, device="cuda")
    z[:, 1] = (torch.arange(T, device="cuda") % 3 - 1).float()
    ids, w = ops.route(z, 1, ids=torch.full((T, 1), -5, dtype=torch.int32, device="cuda"))
    assert torch.equal(ids[:, 0], (z[:, 1] > 0).to(torch.int32))
    assert bool((w == 1).all())


def test_combine():
    """2^35 columns and a few, eight to a thread."""
    T, H = (1 << 23) + 1, 4096
    y = torch.empty(T, H, dtype=BF, device="cuda").fill_(1.5)
    y[-3:], y[: 1 << 10] = 7.0, 3.0
    w = torch.full((T, 1), 2.0, dtype=F32, device="cuda")
    out = torch.empty(T, H, dtype=BF, device="cuda").fill_(float("nan"))
    ops.combine(y, w, out_bf16=out)
    for t in range(0, T, 1 << 20):
        assert torch.equal(out[t:t + (1 << 20)], y[t:t + (1 << 20)] * 2), t


@pytest.mark.parametrize("post", [False, True])
def test_norms(post):
    """2^24 rows and a few, one to a block of 256 threads."""
    T, H = (1 << 24) + 5, 7
    x = torch.empty(T, H, dtype=BF, device="cuda").fill_(-2.0)
    x[:: 5] = 4.0
    w = torch.arange(1, H + 1, device="cuda").float()
    want = x.sign() * w.to(BF)  # a row of equal values has itself as its root mean square
    if post:
        n, _, _ = ops.post_norm(x, w, torch.zeros_like(x), eps=1e-30,
                                out=torch.full_like(x, float("nan")))
    else:
        n, _ = ops.pre_norm(x, w, eps=1e-30)
    assert torch.equal(n, want)

"""Products whose tiles are more than one grid holds: fewer than 2^32 threads (the
runtime runs a grid with more without an error, but only what is left of its threads
behind 32 bits).  The arrays are large, their contents simple."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_grouped_matmul_of_one_k_block():
    """One row for each of 1024 experts, 21900 tiles of 128 columns: 1024 x 8 x 2803200 of
    b, K in one block."""
    E, K, N = 1024, 8, 128 * 21900
    g = torch.Generator("cuda")
    g.manual_seed(1)
    ids = torch.randperm(E, generator=g, device="cuda").to(torch.int32).view(E, 1)
    a = torch.randn(E, K, generator=g, device="cuda").to(BF)
    one = torch.randn(K, N, generator=g, device="cuda").to(BF)
    b = torch.empty(E, K, N, dtype=BF, device="cuda")
    b.copy_(one.expand(E, K, N))
    out = torch.full((E, N), float("nan"), dtype=BF, device="cuda")
    ops.grouped_matmul(a, b, ops.align(ids, E, 16), 1, pair_rows=True, trans=True, out=out)
    for n in range(0, N, 128 * 730):
        w = one[:, n:n + 128 * 730].double()
        ref, mag = a.double() @ w, a.double().abs() @ w.abs()
        bad = (out[:, n:n + 128 * 730].double() - ref).abs() > ref.abs() * R.BF16 + 33 * R.U32 * mag
        nan = torch.isnan(out[:, n:n + 128 * 730])
        assert not bad.any() and not nan.any(), (n, int(bad.sum()), int(nan.sum()))


def test_grouped_wgrad():
    """1024 matrices of 8 x 2097160: 16385 tiles each."""
    E, N, K = 1024, 8, (1 << 21) + 8
    g = torch.Generator("cuda")
    g.manual_seed(2)
    ids = torch.tensor([[1023], [5], [700]], dtype=torch.int32, device="cuda")
    x = torch.randn(3, K, generator=g, device="cuda").to(BF)
    dy = torch.randn(3, N, generator=g, device="cuda").to(BF)
    dw = torch.empty(E, N, K, dtype=BF, device="cuda").fill_(float("nan"))
    ops.grouped_wgrad(dy, x, ops.align(ids, E, 16), 1, out_dtype=BF, out=dw)
    for e, t in ((1023, 0), (5, 1), (700, 2)):
        ref = dy[t].double().unsqueeze(1) * x[t].double()
        assert ((dw[e].double() - ref).abs() <= ref.abs() * R.BF16).all(), e
        dw[e] = 0
    for e in range(0, E, 64):
        assert not dw[e:e + 64].any(), e  # (NaN counts as a value)

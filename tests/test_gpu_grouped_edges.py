"""Far ends of the experts' bf16 products: factors whose product alone leaves fp32's
range."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.mark.parametrize("dt", [BF, F32])
def test_silu_gradient_of_factors_far_apart(dt):
    """d, u and SiLU's slope multiply to numbers in range, two of them alone do not: the
    result is the formula's, as long as the slope is a normal number; behind that it is
    finite."""
    E, k, N, K = 1, 1, 16, 8
    d = [1e30, 1e-30, 1e38, 1.0, 1e30, 1e20, 1e38, 1e-20, 1e-20, 1e30, 3e38, -1e38]
    g = [-60., -60., -86., -80., -80., -80., -30., -85., -80., -200., -1e4, -3e38]
    u = [1e20, 1e38, 1e30, 3.0, 1e-20, -1e38, 1e10, 1e38, 1e30, 1e30, 3e38, 1e38]
    T = len(d)
    a = torch.zeros(T, K, dtype=BF, device="cuda")
    a[:, 0] = torch.tensor(d, device="cuda").to(BF)
    b = torch.zeros(E, K, N, dtype=BF, device="cuda")
    b[:, 0] = 1.0
    gu = torch.empty(T, 2 * N, dtype=BF, device="cuda")
    gu[:, :N] = torch.tensor(g, device="cuda").to(BF).unsqueeze(1)
    gu[:, N:] = torch.tensor(u, device="cuda").to(BF).unsqueeze(1)
    al = ops.align(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), E, 16)
    got = ops.grouped_matmul(a, b, al, k, pair_rows=True, trans=True, act="silu_mul_backward",
                             gu=gu, out_dtype=dt)
    assert torch.isfinite(got).all(), got[:, ::N]
    n = 9  # the rows whose slope is a normal number
    dd, (gg, uu) = a[:n, :1].double(), gu[:n].double().chunk(2, 1)
    s, o = torch.sigmoid(gg), torch.sigmoid(-gg)
    ref = torch.cat([dd * uu * (s * (1 + gg * o)), dd * (gg * s)], 1)
    assert (ref.abs() < 3e38).all()
    # an exponential (two half steps) and at most ten roundings; 1 + g (1 - s) has terms of
    # at most 1.04 times its value at these gates
    tol = ref.abs() * (R.half_step(dt) + 16 * R.U32) + R.TINY
    bad = (got[:n].double() - ref).abs() > tol
    assert not bad.any(), (got[:n, ::N], ref[:, ::N])


def test_a_gate_that_is_no_number_stays_in_its_place():
    """dg and du at that gate are no numbers, and no other value is."""
    T, N, K = 20, 24, 16
    g = torch.Generator("cuda")
    g.manual_seed(3)
    a, b = (torch.randn(*s, generator=g, device="cuda").to(BF) for s in ((T, K), (1, K, N)))
    gu = torch.randn(T, 2 * N, generator=g, device="cuda").to(BF)
    gu[5, 7] = float("nan")
    al = ops.align(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1, 16)
    got = ops.grouped_matmul(a, b, al, 1, pair_rows=True, trans=True, act="silu_mul_backward",
                             gu=gu)
    bad = torch.zeros(T, 2 * N, dtype=torch.bool, device="cuda")
    bad[5, 7] = bad[5, N + 7] = True
    assert torch.equal(torch.isnan(got), bad) and torch.isfinite(got[~bad]).all()

"""The quantizer's SiLU(gate) * up over the whole range of finite gates."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops
from test_gpu_block_ops import _check_groups

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# where the power of two of the sigmoid is 2^100, overflows fp32, or is beyond
# any float; where the argument's product with log2 e overflows; small ones
GATES = [-3.3e38, -2.5e38, -1e30, -1001.0, -999.0, -200.0, -150.0, -110.0, -104.0, -100.0, -95.0,
         -92.0, -90.0, -89.0, -88.75, -88.0, -87.5, -87.34, -87.0, -80.0, -69.5, -69.0, -30.0,
         -1e-3, 1e-3, 20.0, 87.0, 100.0, 127.0, 129.0, 1e4, 1e30, 2.3e38, 2.4e38, 2.5e38, 3.3e38]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("up", [1e-3, 1.0, 1e30, 3e38])
def test_silu_mul_of_any_finite_gate(dtype, up):
    """One gate per group of 128 (SiLU makes the group), with up values of
    sizes from up / 16 to up in both signs."""
    K = 384
    gates = torch.tensor(GATES, device="cuda")
    g = torch.Generator("cuda")
    g.manual_seed(1)
    u = up * ((1 + 15 * torch.rand(len(GATES), K, generator=g, device="cuda")) / 16)
    u = u * (torch.rand(len(GATES), K, generator=g, device="cuda") < 0.5).float().mul(2).sub(1)
    x = torch.cat([gates.unsqueeze(1).expand(-1, K), u], 1).to(dtype)
    v = R.silu_mul(x)
    # exponent, reciprocal and products as at ordinary gates, two more products
    err = 10 * R.U32
    fits = v.abs().amax(1) * (1 + err) <= torch.finfo(F32).max
    assert fits.sum() >= 25  # all but the gates whose product passes fp32
    x, v = x[fits].contiguous(), v[fits]
    v32 = v.float().double()  # as fp32 holds it, which is what is quantized
    r = ops.fp8_quant(x, act="silu_mul")
    assert r["scale"].isfinite().all()
    _check_groups(r["codes"], r["scale"], v32, 1, err)
    both = ops.fp8_quant(x, act="silu_mul", cols=True)
    assert torch.equal(both["codes"], r["codes"]) and torch.equal(both["scale"], r["scale"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_silu_mul_of_gates_that_are_not_finite(dtype):
    """A row with an infinite or NaN gate has a NaN scale in that group only."""
    x = torch.ones(4, 512, dtype=dtype, device="cuda")
    x[0, 3], x[1, 130], x[2, 255] = float("nan"), -float("inf"), float("inf")
    r = ops.fp8_quant(x, act="silu_mul")
    bad = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[1, 2] = True
    assert torch.equal(r["scale"].isnan(), bad)

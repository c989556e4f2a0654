"""How exact the sums of a 4-bit product are: a sum's error is a fraction of the
magnitudes that are summed, whatever x holds where a code is 0.

Tolerance: a code and x are exact in bf16, their products in fp32.  A group's sum is
group additions, each off by at most half a step (2^-24) of S = sum |x q|; one addition
per group and at most 32 for the joining of waves and parts follow, all of them on
values of at most S = sum s |x q|: (group + K / group + 32) 2^-24 S.  Where S is 0 the
result is 0."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=F64)
FORMATS = [(32, False), (64, False), (128, False), (32, True)]
# M, N, K / group: every kernel and choice of them, tails of a K step, a K split
SIZES = [(1, 333, 5), (1, 14000, 9), (4, 4096, 32), (7, 500, 12), (16, 8000, 3), (12, 10300, 4),
         (40, 1000, 6), (130, 512, 7), (300, 4100, 4), (100, 512, 64)]


def _weights(q, scale, group, mx):
    """Values of codes q [N, K] with their scales, in 64 bits."""
    v = E2M1.to(q.device)[q] if mx else ((q + 8) % 16 - 8).double()
    s = torch.exp2(scale.double() - 127) if mx else scale.double()
    return (v.view(q.shape[0], -1, group) * s.unsqueeze(2)).view(q.shape)


def _pack(q):
    return (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8)


def _make(M, N, K, group, mx, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda")
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda")
    if mx:
        scale = torch.randint(117, 125, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    else:
        scale = (torch.rand(N, K // group, generator=g, device="cuda") * 0.02 + 0.001).half()
    return x, q, scale, g


@pytest.mark.parametrize("group,mx", FORMATS)
@pytest.mark.parametrize("M,N,kg", SIZES)
def test_error_follows_what_is_summed(M, N, kg, group, mx):
    """Groups of zeros alone, and channels of x that are 2^30 times the others where
    most weight rows have a code of 0."""
    K = kg * group
    print(f"w4 sums {M} {N} {K} group {group} mxfp4 {mx}", flush=True)
    x, q, scale, g = _make(M, N, K, group, mx, M + N)
    large = torch.rand(K, generator=g, device="cuda") < 0.05
    large[3] = True
    x = torch.where(large, x * 2.0 ** 30, x).to(BF)
    uses = torch.rand(N, 1, generator=g, device="cuda") < 0.25
    q = torch.where(large & ~uses, torch.zeros_like(q), q)
    none = torch.rand(N, kg, generator=g, device="cuda") < 0.3
    none[::7] = True
    q = torch.where(none.repeat_interleave(group, 1), torch.zeros_like(q), q)
    w = _weights(q, scale, group, mx)
    ref, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    assert int((mag == 0).sum()) >= M * (N // 7)
    for dt in (F32, BF):
        got = ops.w4_matmul(x, _pack(q), scale, out_dtype=dt)
        tol = (group + K // group + 32) * R.U32 * mag + ref.abs() * R.half_step(dt)
        bad = (got.double() - ref).abs() > tol
        assert not bad.any(), (dt, int(bad.sum()), float((got.double() - ref)[bad].abs().max()))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 4, 20, 200])
def test_codes_are_exact_in_every_group(M, group):
    """One value of x, one code per weight row, at places all over a group: products of
    8-bit and 4-bit numbers and a scale of one bit are exact."""
    K = 2 * group
    for at in (0, 5, group - 1, group + 7, 2 * group - 2):
        x = torch.zeros(M, K, dtype=BF, device="cuda")
        x[:, at] = (1 + torch.arange(M, device="cuda") / 128).to(BF)
        q = torch.zeros(256, K, dtype=torch.long, device="cuda")
        q[:, at] = torch.arange(256, device="cuda") % 16
        scale = torch.full((256, 2), 2.0 ** -10, dtype=torch.float16, device="cuda")
        scale[128:] = 2.0 ** -24
        ref = x.double() @ _weights(q, scale, group, False).t()
        got = ops.w4_matmul(x, _pack(q), scale, out_dtype=F32)
        assert torch.equal(got.double(), ref), at


@pytest.mark.parametrize("group,mx", FORMATS)
@pytest.mark.parametrize("M", [2, 16, 50, 200])
def test_what_is_not_finite_follows_the_formula(M, group, mx):
    """inf times a code is an infinity of its sign, times 0 no number; opposite
    infinities are no number; other rows stay as they are."""
    N, K = 200, 3 * group
    x, q, scale, _ = _make(M, N, K, group, mx, 5)
    x = x.to(BF)
    x[0, 5] = float("inf")
    x[1, 7], x[1, K - 1] = float("-inf"), float("inf")
    w = _weights(q, scale, group, mx)
    want = x.double() @ w.t()
    two = x[:2, :, None].double() * w.t()  # the terms, each by itself
    plus, minus = (two == float("inf")).any(1), (two == -float("inf")).any(1)
    no = torch.isnan(two).any(1) | (plus & minus)
    got = ops.w4_matmul(x, _pack(q), scale, out_dtype=F32)
    assert torch.equal(torch.isnan(got[:2]), no)
    assert torch.equal(got[:2] == float("inf"), plus & ~no)
    assert torch.equal(got[:2] == -float("inf"), minus & ~no)
    assert torch.isfinite(got[2:]).all()
    mag = x[2:].double().abs() @ w.abs().t()
    assert ((got[2:].double() - want[2:]).abs() <= (group + 35) * R.U32 * mag + R.U32
            * want[2:].abs()).all()

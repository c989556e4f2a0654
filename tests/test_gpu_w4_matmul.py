"""Dense products with 4-bit weights against plain forms in 64 bits.

Tolerances: the values of codes and x are exact in bf16 and their products in
fp32.  int4 weights enter as 1.5 + q / 16 (at most 2, against |q| / 16 <= 1/2) and
-1.5 times the sum of x is where the sum starts, so that a group's sum passes
through values of at most 3.5 X with X = sum |x| over the group: two times (group
/ 32) instructions of 32 products, each within 32 half steps of that, 16 times
the scale; then one addition per group and the joining of the parts.  In all
((group / 16) * 32 * 3.5 * 16 s X + (K / group + 32) S) 2^-24 with S the sum of
magnitudes s |x q|; an e2m1 group's sum is within 32 half steps of S's."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=F64)


def _make(M, N, K, group, mx, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if mx:
        scale = torch.randint(117, 125, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    else:
        scale = (torch.rand(N, K // group, generator=g, device="cuda") * 0.02 + 0.001).half()
    return x, codes, scale


def _plain(x, codes, scale, group, mx):
    """(products, tolerance of the fp32 sums) in 64 bits."""
    N, K = codes.shape[0], 2 * codes.shape[1]
    q = torch.stack([codes & 15, codes >> 4], 2).view(N, K).long()
    if mx:
        v, s = E2M1.to(q.device)[q], torch.exp2(scale.double() - 127)
    else:
        v, s = ((q + 8) % 16 - 8).double(), scale.double()
    w = (v.view(N, K // group, group) * s.unsqueeze(2)).view(N, K)
    y, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    tol = (K // group + 32) * R.U32 * mag
    if mx:
        tol = tol + 32 * R.U32 * mag
    else:
        X = x.double().abs().view(x.shape[0], K // group, group).sum(2)
        tol = tol + group / 16 * 32 * 3.5 * 16 * R.U32 * (X @ s.t())
    return y, tol


def _check(got, ref, tol, what=None):
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float((got.double() - ref).abs().max()))


FORMATS = [(32, False), (64, False), (128, False), (32, True)]
# M, N, K in units of the group: tails of the K step, odd columns, both sides of every
# choice of kernel
SIZES = [(1, 1, 1), (1, 40, 3), (2, 1000, 33), (5, 17, 8), (16, 333, 5), (17, 64, 12), (33, 130, 7),
         (64, 48, 4), (65, 257, 9), (130, 512, 6), (300, 129, 10), (1, 4096, 32), (257, 1024, 16),
         (2, 12300, 2), (8, 7000, 3), (9, 10300, 3), (50, 7000, 9), (130, 16400, 4), (100, 512, 64)]


@pytest.mark.parametrize("group,mx", FORMATS)
@pytest.mark.parametrize("M,N,kg", SIZES)
def test_w4_matmul(M, N, kg, group, mx):
    K = kg * group
    print(f"w4 {M} {N} {K} group {group} mxfp4 {mx}", flush=True)
    x, codes, scale = _make(M, N, K, group, mx, M + N)
    ref, tol = _plain(x, codes, scale, group, mx)
    for dt in (BF, F32):
        got = ops.w4_matmul(x, codes, scale, out_dtype=dt)
        _check(got, ref, ref.abs() * R.half_step(dt) + tol, dt)
        add = torch.randn(M, N, device="cuda").to(dt)
        want = ref + add.double()
        t = want.abs() * R.half_step(dt) + tol + 2 * R.U32 * (ref.abs() + add.double().abs())
        _check(ops.w4_matmul(x, codes, scale, add=add, out_dtype=dt), want, t, "add")
        out = add.clone()
        assert ops.w4_matmul(x, codes, scale, add=out, out=out, out_dtype=dt) is out
        _check(out, want, t, "in place")
        assert torch.equal(got, ops.w4_matmul(x, codes, scale, out_dtype=dt))


@pytest.mark.parametrize("group,mx", FORMATS)
@pytest.mark.parametrize("M,N,kg", [(1, 2, 1), (1, 768, 16), (5, 90, 9), (16, 1024, 5), (40, 34, 8),
                                    (130, 386, 7), (300, 512, 4), (100, 512, 64),
                                    (12, 14000, 5), (200, 33000, 2)])
def test_w4_silu_mul(M, N, kg, group, mx):
    K = kg * group
    print(f"w4 silu_mul {M} {N} {K} group {group} mxfp4 {mx}", flush=True)
    x, codes, scale = _make(M, N, K, group, mx, M + 2 * N)
    y, t = _plain(x, codes, scale, group, mx)
    (g, u), (eg, eu) = y.chunk(2, 1), t.chunk(2, 1)
    s = g * torch.sigmoid(g)
    ref = s * u
    err = 1.1 * u.abs() * eg + s.abs() * eu + 1.1 * eg * eu + 8 * R.U32 * ref.abs()
    add = torch.randn(M, N // 2, device="cuda")
    for dt in (BF, F32):
        got = ops.w4_matmul(x, codes, scale, act="silu_mul", out_dtype=dt)
        _check(got, ref, ref.abs() * R.half_step(dt) + err * 1.01, dt)
        want = ref + add.to(dt).double()
        got = ops.w4_matmul(x, codes, scale, act="silu_mul", add=add.to(dt), out_dtype=dt)
        _check(got, want, want.abs() * R.half_step(dt) + err * 1.01
               + 2 * R.U32 * (ref.abs() + add.double().abs()), "add")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M", [1, 20, 200])
def test_every_code_and_scale(M, mx):
    """One group per output: each code alone, each power of two as an e8m0 scale,
    fp16's smallest and largest scales."""
    N, K = 256, 32
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[:, 3] = 2.0 ** torch.arange(M, device="cuda").remainder(8).to(F32)
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    n = torch.arange(N, device="cuda")
    codes[:, 1] = (n % 16 * 16).to(torch.uint8)  # code n % 16 at K 3, others 0
    if mx:
        scale = n.clamp(0, 244).to(torch.uint8).view(N, 1)  # up to 2^117: finite with x and 6
    else:
        scale = torch.full((N, 1), 2.0 ** -24, dtype=torch.float16, device="cuda")
        scale[128:] = 65504.0
    ref, _ = _plain(x, codes, scale, 32, mx)
    got = ops.w4_matmul(x, codes, scale, out_dtype=F32)
    if mx:  # exact, but for products below fp32's normal numbers, which may be flushed
        small = ref.abs() < R.TINY
        assert torch.equal(got.double()[~small], ref[~small])
        assert (got.double()[small] - ref[small]).abs().max() <= R.TINY
    else:
        assert torch.equal(got.double(), ref)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M", [1, 16, 50, 200])
def test_what_lies_behind_is_not_used(M, mx):
    """Rows, codes and scales end where NaN begins; a row of x that is not finite
    stays in its row."""
    N, group, K = 100, 32, 32 * 7
    x, codes, scale = _make(M, N, K, group, mx, 3)
    ref, tol = _plain(x, codes, scale, group, mx)
    px = torch.full((M * K + 4096,), float("nan"), dtype=BF, device="cuda")
    px[:M * K] = x.view(-1)
    pc = torch.full((codes.numel() + 4096,), 0x77, dtype=torch.uint8, device="cuda")
    pc[:codes.numel()] = codes.view(-1)
    ps = torch.full((scale.numel() + 4096,), float("nan"), dtype=F32, device="cuda").to(
        torch.float16) if not mx else torch.full((scale.numel() + 4096,), 255, dtype=torch.uint8,
                                                 device="cuda")
    ps[:scale.numel()] = scale.view(-1)
    po = torch.full((M * N + 4096,), 5.0, dtype=BF, device="cuda")
    out = po[:M * N].view(M, N)
    ops.w4_matmul(px[:M * K].view(M, K), pc[:codes.numel()].view_as(codes),
                  ps[:scale.numel()].view_as(scale), out=out)
    _check(out, ref, ref.abs() * R.BF16 + tol)
    assert (po[M * N:] == 5.0).all()
    if M > 1:
        x[1, 5] = float("inf")
        got = ops.w4_matmul(x, codes, scale)
        keep = torch.arange(M, device="cuda") != 1
        _check(got[keep], ref[keep], (ref.abs() * R.BF16 + tol)[keep])
        assert not torch.isfinite(got[1]).any()


def test_an_experts_matrix_of_the_layer():
    """int4 groups of 32 are the W4A16 scheme's canonical layout: one expert's
    gate/up and down products equal the layer with that expert alone, up to the
    layer's own roundings (weights and h to bf16)."""
    from quantized_mixture_experts_moe_amd import synth
    from quantized_mixture_experts_moe_amd.shapes import W4A16_TINY as sh
    from _helpers import gpu_inputs
    inp = gpu_inputs(synth.make_inputs(sh))
    w = {n: inp[n][:1].contiguous() for n in ("w13", "w13_scale", "w2", "w2_scale")}
    x = inp["x"]
    T = x.shape[0]
    r = ops.moe_forward("w4a16", torch.zeros(T, 1, device="cuda"), x, None, w, 1, 16)
    h = ops.w4_matmul(x, w["w13"][0], w["w13_scale"][0].view(torch.float16), act="silu_mul")
    y = ops.w4_matmul(h, w["w2"][0], w["w2_scale"][0].view(torch.float16))
    d = (y.double() - r["out"].double()).norm() / r["out"].double().norm()
    # a rounding to bf16 is off by up to 2^-8 2^e, 2^-8 / sqrt(3) = 2.26e-3 in the mean square
    # of a value of 2^e.  Seven of them: gate's weights, up's, w2's, and h and y on both
    # sides; independent, so sqrt(7) * 2.26e-3 = 6.0e-3
    assert float(d) <= 6.0e-3


def test_no_rows():
    x, codes, scale = _make(0, 64, 128, 32, False, 1)
    assert ops.w4_matmul(x, codes, scale).shape == (0, 64)
    assert ops.w4_matmul(x, codes, scale, act="silu_mul").shape == (0, 32)

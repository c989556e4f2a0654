"""Norms and their gradients at the ends of the activations' range, against
their 64-bit forms."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
EPS32 = float(torch.tensor(EPS))  # what the fp32 argument holds


def _rand(*shape, seed=0, scale=1.0, dtype=F32):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _large(T, H, dtype, seed):
    """Rows from ordinary ones to 1e36, whose squares fp32 does not hold."""
    sizes = torch.tensor([1.0, 1e18, 3e19, 1e20, 1e25, 1e36], device="cuda")
    x = _rand(T, H, seed=seed)
    return (x * sizes[torch.arange(T, device="cuda") % 6].unsqueeze(1)).to(dtype)


# every shape of the kernels: threads per row, vectors per thread, scalar loads
WIDTHS = [64, 200, 512, 1000, 2048, 4096, 777, 8192, 8191, 16384]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_rows_whose_squares_pass_fp32(H, dtype):
    T = 13
    x, w = _large(T, H, dtype, H), 1 + 0.3 * _rand(H, seed=2)
    ref = R.norm(x.double(), w.double(), EPS32)
    # r, the product with it, the product with w: half a step each, and one more
    # for their products
    n, _ = ops.pre_norm(x, w, eps=EPS, out="f32")
    assert ((n.double() - ref).abs() <= ref.abs() * 4 * R.U32 + R.TINY).all()
    out, _, _ = ops.post_norm(x, w, torch.zeros_like(x), eps=EPS)
    assert ((out.double() - ref).abs()
            <= ref.abs() * (4 * R.U32 + R.half_step(dtype)) + R.TINY).all()

    d = _rand(T, H, seed=4, dtype=dtype)
    gate = torch.sigmoid(_rand(T, 1, seed=6))
    v64, d64 = x.double(), d.double()
    r = 1 / torch.sqrt((v64 * v64).mean(1, keepdim=True) + EPS32)
    h = v64 * r
    # sums of H terms in fp32: chains of 32 and 12 steps, as many half steps of
    # the magnitudes' sum; a handful of products besides
    tol_sum, few = 44 * R.U32, 12 * R.U32

    def check(dv, dh):
        want = r * (dh - h * (dh * h).mean(1, keepdim=True))
        size = r * (dh.abs() + h.abs() * (dh * h).abs().mean(1, keepdim=True))
        tol = size * (2 * tol_sum + few)
        assert ((dv.double() - want).abs()
                <= tol + (want.abs() + tol) * R.half_step(dtype) + R.TINY).all()

    def check_sum(dw, terms):
        assert ((dw.double() - terms.sum(0)).abs()
                <= terms.abs().sum(0) * (tol_sum + few) + 1e-37).all()

    dx, dw = ops.pre_norm_backward(d, x, w, eps=EPS)
    check(dx, d64 * w.double())
    check_sum(dw, d64 * h)
    b = ops.post_norm_backward(d, x, w, gate=gate, alpha=0.5, eps=EPS)
    check(b["dy"], d64 * gate.double() * w.double())
    check_sum(b["dw"], d64 * gate.double() * h)
    terms = d64 * h * w.double()
    assert ((b["dgate"].double() - terms.sum(1, keepdim=True)).abs()
            <= terms.abs().sum(1, keepdim=True) * (tol_sum + few)).all()


@pytest.mark.parametrize("H", [512, 777, 4096])
def test_rows_of_other_sizes_keep_their_gradients(H):
    """A large row changes nothing in the other rows of its block."""
    x, w, d = _rand(8, H, seed=1), 1 + 0.3 * _rand(H, seed=2), _rand(8, H, seed=3)
    dx, _ = ops.pre_norm_backward(d, x, w)
    y = ops.post_norm_backward(d, x, w)["dy"]
    x[5] *= 1e30
    rest = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(ops.pre_norm_backward(d, x, w)[0][rest], dx[rest])
    assert torch.equal(ops.post_norm_backward(d, x, w)["dy"][rest], y[rest])


# ---------------------------------------------------------------- the stored out

def _bf16(v):
    """v (float64) as fp32 holds it, rounded to bf16 (8 significant bits, ties to
    even): what a conversion of the 64-bit value gives."""
    v = v.float().double()
    step = torch.exp2(torch.frexp(v).exponent.double() - 8)
    return torch.round(v / step) * step


@pytest.mark.parametrize("T,H", [(3000, 333), (2000, 512), (1000, 1000), (1030, 2048), (300, 4096),
                                 (130, 8192), (67, 16384), (150, 8191)])
@pytest.mark.parametrize("cancel", [False, True])
def test_bf16_out_is_rounded_once(T, H, cancel):
    """out is the definition's value, as fp32 holds it, in bf16, so what the next norm
    makes of it in fp32 (n, scales) is off by fp32 steps, not by bf16 ones.
    cancel: x takes away most of the gated norm."""
    y, w, w2 = _rand(T, H, seed=H), 1 + 0.3 * _rand(H, seed=2), 1 + 0.3 * _rand(H, seed=3)
    y = (y * torch.exp(_rand(T, 1, seed=5))).to(BF)
    gates = [None, 0.5 + _rand(H, seed=11), torch.sigmoid(_rand(T, 1, seed=12)),
             torch.sigmoid(_rand(T, H, seed=13)).to(BF)]
    forms = ["f32", "e4m3_128", "e4m3", "int8"]
    for i, gate in enumerate(gates):
        alpha = (1.0, 0.3, -0.5, 0.7)[i]
        al32 = float(torch.tensor(alpha))
        u = R.norm(y.double(), w.double(), EPS32) * (1.0 if gate is None else gate.double())
        x = (-u / alpha if cancel else _rand(T, H, seed=9) * 2).to(BF)
        want = _bf16(al32 * x.double() + u)
        out, _, _ = ops.post_norm(y, w, x, gate=gate, alpha=alpha, eps=EPS)
        bad = out.double() != want
        assert not bad.any(), f"gate {i}: {int(bad.sum())} of {bad.numel()}"
        o2, n, scale = ops.post_norm(y, w, x, gate=gate, alpha=alpha, eps=EPS, next_weight=w2,
                                     next_out=forms[i])
        assert torch.equal(o2, out)
        ref = R.norm(want, w2.double(), EPS32)
        # r, v r and the product with w: half a step each, and one for their products
        rel = 4 * R.U32
        if forms[i] == "f32":
            assert ((n.double() - ref).abs() <= ref.abs() * rel + R.TINY).all()
        else:
            g = R.pad_to(ref, R.up128(H), 1).view(T, -1, 128) if forms[i] == "e4m3_128" \
                else ref.view(T, 1, H)
            s = R.group_scale(g.abs().amax(2), 127.0 if forms[i] == "int8" else 448.0)
            got = scale.t() if forms[i] == "e4m3_128" else scale.view(T, 1)
            assert ((got.double() - s).abs() <= s * (rel + R.U32)).all()

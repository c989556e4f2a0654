"""The layer with bf16 experts as it is trained, forward and backward: routing,
the experts' products, the routed sum, the balance loss' gradient, and every
gradient; on streams and in graphs; with a 4-bit shared expert beside it."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def _rand(*shape, seed=0, scale=1.0, dtype=BF):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _layer(T, H, I, E, k, seed=0):
    w = {"w13": _rand(E, 2 * I, H, seed=seed, scale=H ** -0.5),
         "w2": _rand(E, H, I, seed=seed + 1, scale=I ** -0.5)}
    return _rand(T, H, seed=seed + 2), _rand(T, E, seed=seed + 3, dtype=F32), w, \
        _rand(T, H, seed=seed + 4)


def _plain(logits, x, w13, w2, ids):
    """The layer in 64 bits for picks that are given."""
    T, k = ids.shape
    w = torch.softmax(logits.gather(1, ids.long()), 1).reshape(-1)
    flat, out = ids.reshape(-1), torch.zeros_like(x)
    for e in range(w13.shape[0]):
        p = (flat == e).nonzero().reshape(-1)
        if p.numel():
            g, u = (x[p // k] @ w13[e].t()).chunk(2, 1)
            y = (g * torch.sigmoid(g) * u) @ w2[e].t()
            out = out.index_add(0, p // k, w[p].unsqueeze(1) * y)
    return out


def _step(x, logits, w, k, dout):
    f = ops.bf16_moe_forward(logits, x, w, k)
    b = ops.balance_loss(logits, f["topk_ids"], coef=0.01)
    dz = ops.balance_loss_backward(logits, b["counts"], b["tokens"], k, torch.ones_like(b["loss"]),
                                   coef=0.01)
    g = ops.bf16_moe_backward(dout, f, x, w, add=dz)
    return {"out": f["out"], "h": f["h"], "loss": b["loss"], "balance": dz, **g}


SIZES = [(1, 256, 128, 8, 2), (17, 64, 40, 5, 3), (64, 256, 128, 8, 2), (300, 384, 264, 6, 4),
         (700, 128, 512, 16, 2)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_layer_against_64_bits(T, H, I, E, k):
    print(f"train {T} {H} {I} {E} {k}", flush=True)
    x, logits, w, dout = _layer(T, H, I, E, k, seed=T)
    r = _step(x, logits, w, k, dout)
    ids = ops.route(logits, k)[0]
    leaf = [t.double().requires_grad_(True) for t in (logits, x, w["w13"], w["w2"])]
    out = _plain(*leaf, ids)
    (out * dout.double()).sum().backward()
    want = {"out": out.detach(), "dlogits": leaf[0].grad + r["balance"].double(),
            "dx": leaf[1].grad, "dw13": leaf[2].grad, "dw2": leaf[3].grad}
    for name, ref in want.items():
        err = float((r[name].double() - ref).norm() / ref.norm())
        # a rounding to bf16 is at most 2^-8 / sqrt(3) = 2.26e-3 off in the mean square; out
        # sees three (h, the experts' outputs, out), the gradients up to six (gate and up as
        # they are kept, h or the outputs' gradient, the gradient of gate/up, the pairs'
        # gradients, the result), where SiLU's slopes turn one of the gate's into at most
        # two of its gradient's: sqrt(4 + 5) * 2.26e-3 = 6.8e-3, and a tenth for T = 1's few values
        assert err <= 7.5e-3, (name, err)


def test_gradients_against_differences():
    """The derivative along random directions of sum(dout * layer), by differences of the
    plain form in 64 bits."""
    T, H, I, E, k = 40, 64, 48, 6, 2
    x, logits, w, dout = _layer(T, H, I, E, k, seed=5)
    f = ops.bf16_moe_forward(logits, x, w, k)
    g = ops.bf16_moe_backward(dout, f, x, w)
    at = [t.double() for t in (logits, x, w["w13"], w["w2"])]
    for i, name in enumerate(("dlogits", "dx", "dw13", "dw2")):
        d = g[name].double()
        step = d / d.norm()  # along the gradient itself: the derivative is its norm
        h = 1e-4

        def value(s):
            return (_plain(*[t + s * step if j == i else t for j, t in enumerate(at)],
                           f["topk_ids"]) * dout.double()).sum()
        slope = float((value(h) - value(-h)) / (2 * h))
        # <d, true> / |d|: the roundings' error (7.5e-3 of the norm) enters this by its part
        # along d alone; differences leave h^2 times the third derivative
        assert abs(slope - float(d.norm())) <= 7.5e-3 * float(d.norm()), name


def test_no_tokens():
    x, logits, w, dout = _layer(0, 64, 32, 4, 2)
    r = _step(x, logits, w, 2, dout)
    assert r["out"].shape == (0, 64) and r["dx"].shape == (0, 64) and r["dlogits"].shape == (0, 4)
    assert not r["dw13"].any() and not r["dw2"].any()


@pytest.mark.parametrize("T", [3, 200])
def test_step_in_graphs_and_on_a_stream(T):
    """Two graphs and an eager step on a stream of its own, replayed on new inputs with
    eager work between, equal the eager step bit for bit."""
    H, I, E, k = 128, 72, 8, 2
    x, logits, w, dout = _layer(T, H, I, E, k, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(x, logits, w, k, dout)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = _step(x, logits, w, k, dout)
        graphs.append((g, r))
    for turn in range(4):
        x.copy_(_rand(T, H, seed=100 + turn))
        logits.copy_(_rand(T, E, seed=200 + turn, dtype=F32))
        dout.copy_(_rand(T, H, seed=300 + turn))
        want = {n: t.clone() for n, t in _step(x, logits, w, k, dout).items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = _step(x, logits, w, k, dout)
        for g, r in graphs:
            g.replay()
        torch.cuda.synchronize()
        for r in [other] + [r for _, r in graphs]:
            for n, t in want.items():
                assert torch.equal(r[n], t), (turn, n)


@pytest.mark.parametrize("T", [1, 6, 90])
def test_shared_expert_beside_the_routed_ones(T):
    """out = the routed experts' sum + a 4-bit shared expert of the same input."""
    H, I, E, k = 256, 128, 8, 2
    x, logits, w, _ = _layer(T, H, I, E, k, seed=T)
    f = ops.bf16_moe_forward(logits, x, w, k)
    g = torch.Generator("cuda")
    g.manual_seed(T)

    def weights(n, kk):
        codes = torch.randint(0, 256, (n, kk // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = (torch.rand(n, kk // 32, generator=g, device="cuda") * 0.01 + 0.005).half()
        return codes, scale, (torch.stack([(codes & 15).int(), (codes >> 4).int()], 2).view(n, kk)
                              .add(8).remainder(16).sub(8).double().view(n, kk // 32, 32)
                              * scale.double().unsqueeze(2)).view(n, kk)

    c13, s13, w13 = weights(2 * I, H)
    c2, s2, w2 = weights(H, I)
    h = ops.w4_matmul(x, c13, s13, act="silu_mul")
    out = ops.w4_matmul(h, c2, s2, add=f["out"])
    a, u = (x.double() @ w13.t()).chunk(2, 1)
    hr = a * torch.sigmoid(a) * u
    assert ((h.double() - hr).abs() <= hr.abs() * R.BF16 + 1e-4 * (u.abs() + a.abs() + 1)).all()
    y = h.double() @ w2.t()
    want = y + f["out"].double()
    assert ((out.double() - want).abs() <= want.abs() * R.BF16
            + 2e-3 * R.BF16 * (h.double().abs() @ w2.abs().t())).all()

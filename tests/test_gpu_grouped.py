"""bf16 products of the experts and their gradients against plain forms in 64
bits.

Tolerances: products of two bf16 numbers are exact in fp32; a sum of n of them
is formed in groups of 16 by one instruction, so that a value passes through at
most n / 16 additions to the running sum and the 16 inside an instruction, each
off by half a step (2^-24) of at most the sum of the magnitudes S, and through
the joining of partial sums: (n / 16 + 32) 2^-24 S in all, plus the half step of
the output's type."""
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


def _ids(T, E, k, seed, skew=False):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    z = torch.randn(T, E, generator=g, device="cuda")
    if skew:  # most rows on a few experts, some experts without a row
        z -= 3.0 * torch.log(torch.arange(1, E + 1, device="cuda").float())
    return z.topk(k, 1).indices.to(torch.int32) if T else torch.empty((0, k), dtype=torch.int32,
                                                                      device="cuda")


def _plain(a, b, ids, pair_rows, trans):
    """(products, sums of magnitudes) [P, N] in 64 bits; rows of bad ids are 0."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    N = b.shape[2] if trans else b.shape[1]
    y = torch.zeros(T * k, N, dtype=F64, device="cuda")
    m = torch.zeros_like(y)
    for e in range(b.shape[0]):
        p = (flat == e).nonzero().reshape(-1)
        if p.numel():
            w = b[e].double() if trans else b[e].double().t()
            x = a[p if pair_rows else p // k].double()
            y[p], m[p] = x @ w, x.abs() @ w.abs()
    return y, m


def _sum_tol(n):
    return (n / 16 + 32) * R.U32


def _close(got, ref, tol, what=""):
    bad = (got.double() - ref).abs() > tol
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    assert not bad.any(), (what, int(bad.sum()), float((got.double() - ref).abs().max()))


# T, E, k, N, K: one token to long segments, experts without rows, sizes that no tile divides
SIZES = [(1, 8, 2, 64, 64), (1, 1, 1, 8, 8), (3, 16, 4, 96, 136), (7, 4, 4, 48, 1000),
         (40, 8, 2, 272, 264), (130, 8, 2, 128, 128), (300, 4, 3, 520, 328), (700, 3, 1, 256, 72),
         (1100, 2, 2, 144, 192), (9, 300, 5, 64, 200),
         # enough tiles for the wide ones and for blocks that take several, K of one and two blocks
         (150, 8, 2, 1040, 200), (700, 16, 2, 4112, 136), (1500, 16, 2, 4112, 72),
         (2200, 16, 2, 4112, 200), (2200, 16, 2, 2064, 64), (700, 2, 1, 4088, 2040),
         (700, 16, 2, 2064, 200), (700, 16, 2, 2064, 72), (1500, 16, 2, 2064, 136),
         (1000, 16, 2, 4080, 64), (1500, 16, 2, 3080, 72)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_matmul(T, E, k, N, K, trans):
    print(f"grouped_matmul {T} {E} {k} {N} {K} trans {trans}", flush=True)
    ids = _ids(T, E, k, T + E, skew=T % 2 == 0)
    b = _rand(E, *((K, N) if trans else (N, K)), seed=1, scale=K ** -0.5)
    for pair_rows in (False, True):
        a = _rand(T * k if pair_rows else T, K, seed=2)
        ref, mag = _plain(a, b, ids, pair_rows, trans)
        for bm in (16, 128):
            al = ops.align(ids, E, bm)
            for dt in (BF, F32):
                got = ops.grouped_matmul(a, b, al, k, pair_rows=pair_rows, trans=trans,
                                         out_dtype=dt)
                assert got.dtype == dt
                _close(got, ref, ref.abs() * R.half_step(dt) + _sum_tol(K) * 1.01 * mag,
                       (pair_rows, bm, dt))


def _silu_grad(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


@pytest.mark.parametrize("T,E,k,N,K", [(t, e, k, (n + 15) // 16 * 16, kk)
                                       for t, e, k, n, kk in SIZES])
def test_silu_mul(T, E, k, N, K):
    print(f"silu_mul {T} {E} {k} {N} {K}", flush=True)
    ids = _ids(T, E, k, 3 * T + E, skew=T % 3 == 0)
    b, a = _rand(E, N, K, seed=3, scale=K ** -0.5), _rand(T, K, seed=4, scale=2.0)
    al = ops.align(ids, E, 16)
    y, mag = _plain(a, b, ids, False, False)
    g, u = y.chunk(2, 1)
    eg, eu = (_sum_tol(K) * 1.01 * mag).chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    # SiLU's slope is below 1.1; its evaluation and the products are within 8 half steps
    err = (1.1 * u.abs() * eg + (g * torch.sigmoid(g)).abs() * eu + 1.1 * eg * eu
           + 8 * R.U32 * ref.abs())
    for dt in (BF, F32):
        gu = torch.full((T * k, N), float("nan"), dtype=BF, device="cuda")
        h = ops.grouped_matmul(a, b, al, k, act="silu_mul", gu=gu, out_dtype=dt)
        _close(h, ref, ref.abs() * R.half_step(dt) + err * 1.01, dt)
        _close(gu, y, y.abs() * R.BF16 + _sum_tol(K) * 1.01 * mag, "gu")
        assert torch.equal(h, ops.grouped_matmul(a, b, al, k, act="silu_mul", out_dtype=dt))


@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_silu_mul_backward(T, E, k, N, K):
    print(f"silu_mul_backward {T} {E} {k} {N} {K}", flush=True)
    ids = _ids(T, E, k, 5 * T + E)
    b, a = _rand(E, K, N, seed=5, scale=K ** -0.5), _rand(T * k, K, seed=6)
    gu = _rand(T * k, 2 * N, seed=7, scale=4.0)
    if T > 1:  # far ends of the gate: the gradient is 0 or up's
        gu[0, :4] = torch.tensor([-3e38, -200.0, 200.0, 3e38], device="cuda").to(BF)
    al = ops.align(ids, E, 16)
    d, mag = _plain(a, b, ids, True, True)
    ed = _sum_tol(K) * 1.01 * mag
    g, u = gu.double().chunk(2, 1)
    f, s = _silu_grad(g), g * torch.sigmoid(g)
    f = torch.where(g < -1e4, torch.zeros_like(f), f)  # (0 times a large number in 64 bits)
    ref = torch.cat([d * u * f, d * s], 1)
    # f: sums of terms of at most 1.3 in all, to 8 half steps; the products 4 more
    err = torch.cat([ed * u.abs() * 1.1 + (d * u).abs() * 12 * 1.3 * R.U32,
                     ed * s.abs() + 12 * R.U32 * (d * s).abs()], 1)
    for dt in (BF, F32):
        got = ops.grouped_matmul(a, b, al, k, pair_rows=True, trans=True, act="silu_mul_backward",
                                 gu=gu, out_dtype=dt)
        # exp(-200) = 1.4e-87 lies below fp32's smallest number, 2^-149: such a result is 0
        # and d * 3e38 beyond the type's largest number (both 3.4e38) where d is above 1.13: it
        # is an infinity of the product's sign
        over = ref.abs() > torch.finfo(dt).max * (1 - 2 * R.half_step(dt))
        assert (got[over].double() * ref[over].sign() > 3e38).all()
        assert int(over.sum()) <= 1
        got[over] = 0
        _close(got, torch.where(over, torch.zeros_like(ref), ref),
               ref.abs() * R.half_step(dt) + err * 1.01 + R.TINY, dt)


@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_wgrad(T, E, k, N, K):
    print(f"wgrad {T} {E} {k} {N} {K}", flush=True)
    ids = _ids(T, E, k, 7 * T + E, skew=T % 2 == 0)
    dy = _rand(T * k, N, seed=8)
    flat = ids.reshape(-1)
    for pair_rows in (False, True):
        x = _rand(T * k if pair_rows else T, K, seed=9)
        ref = torch.zeros(E, N, K, dtype=F64, device="cuda")
        mag, rows = torch.zeros_like(ref), torch.zeros(E, 1, 1, dtype=F64, device="cuda")
        for e in range(E):
            p = (flat == e).nonzero().reshape(-1)
            xs, ds = x[p if pair_rows else p // k].double(), dy[p].double()
            ref[e], mag[e], rows[e] = ds.t() @ xs, ds.abs().t() @ xs.abs(), p.numel()
        tol = (rows / 16 + 32) * R.U32 * mag
        for bm in (16, 64):
            al = ops.align(ids, E, bm)
            for dt in (BF, F32):
                got = ops.grouped_wgrad(dy, x, al, k, pair_rows=pair_rows, out_dtype=dt)
                _close(got, ref, ref.abs() * R.half_step(dt) + tol, (pair_rows, bm, dt))
                assert not got[rows.view(-1) == 0].any()
        was = _rand(E, N, K, seed=10, dtype=F32)
        acc = was.clone()
        assert ops.grouped_wgrad(dy, x, al, k, pair_rows=pair_rows, out=acc,
                                 accumulate=True) is acc
        _close(acc, ref + was.double(), (ref.abs() + was.double().abs()) * 2 * R.U32 + tol, "acc")


@pytest.mark.parametrize("T", [0, 1, 5, 200])
def test_dropped_pairs(T):
    """Pairs whose id no expert has: rows left as they are, nothing in dw."""
    E, k, N, K = 6, 3, 64, 72
    ids = _ids(T, E, k, 11)
    if T:
        ids[0, 0], ids[T // 2, 2] = E + 5, -1
    al = ops.align(ids, E, 16)
    gone = ((ids < 0) | (ids >= E)).reshape(-1)
    a, b = _rand(T, K, seed=1), _rand(E, N, K, seed=2)
    a[:, 0] = float("inf") if T == 0 else a[:, 0]
    out = torch.full((T * k, N), 7.0, dtype=BF, device="cuda")
    ops.grouped_matmul(a, b, al, k, out=out)
    ref, mag = _plain(a, b, ids, False, False)
    assert (out[gone] == 7.0).all()
    _close(out[~gone], ref[~gone], (ref.abs() * R.BF16 + _sum_tol(K) * 1.01 * mag)[~gone])
    dy = _rand(T * k, N, seed=3)
    dy[gone] = float("nan")
    dw = ops.grouped_wgrad(dy, a, al, k)
    want = torch.zeros(E, N, K, dtype=F64, device="cuda")
    for e in range(E):
        p = (ids.reshape(-1) == e).nonzero().reshape(-1)
        want[e] = dy[p].double().t() @ a[p // k].double()
    assert torch.isfinite(dw).all() and (dw.double() - want).abs().max() <= 1e-3 if T else \
        not dw.any()


@pytest.mark.parametrize("T", [4, 300])
def test_what_is_not_finite_stays_in_its_row(T):
    """A row of a or of an expert's matrix that is not finite reaches the outputs
    of that row or column, and no other; memory behind the operands holds NaN."""
    E, k, N, K = 4, 2, 80, 88
    ids = _ids(T, E, k, 12)
    al = ops.align(ids, E, 16)
    pool = torch.full((1 << 21,), float("nan"), dtype=BF, device="cuda")
    a = pool[:T * K].view(T, K)
    a.copy_(_rand(T, K, seed=1))
    b = pool[1 << 20:][:E * N * K].view(E, N, K)
    b.copy_(_rand(E, N, K, seed=2))
    a[T // 2] = float("nan")
    b[1, 5] = float("inf")
    for trans in (False, True):
        w = b if not trans else b.transpose(1, 2).contiguous()
        got = ops.grouped_matmul(a, w, al, k, trans=trans).view(T, k, N)
        bad = torch.zeros(T, k, N, dtype=torch.bool, device="cuda")
        bad[T // 2] = True
        bad[:, :, 5] |= ids == 1
        assert torch.isfinite(got[~bad]).all()
        assert not torch.isfinite(got[bad]).any()
    dy = _rand(T * k, N, seed=3)
    dy[0, 3] = float("nan")
    dw = ops.grouped_wgrad(dy, torch.nan_to_num(a), al, k)
    e = int(ids[0, 0])
    assert torch.isnan(dw[e, 3]).all()
    dw[e, 3] = 0
    assert torch.isfinite(dw).all()


# ---------------------------------------------------------------- the routed sum's gradient

@pytest.mark.parametrize("T,E,k,H", [(1, 4, 1, 8), (5, 8, 2, 256), (64, 8, 8, 512),
                                     (33, 60, 4, 520),
                                     (257, 512, 10, 2048), (3, 1024, 16, 4096), (130, 17, 5, 1000)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_combine_backward(T, E, k, H, dt):
    print(f"combine_backward {T} {E} {k} {H} {dt}", flush=True)
    logits = _rand(T, E, seed=1, dtype=F32)
    ids, w = ops.route(logits, k)
    y, dout = _rand(T * k, H, seed=2, dtype=dt), _rand(T, H, seed=3, dtype=dt)
    add = _rand(T, E, seed=4, dtype=F32)
    wd, dd, yd = w.double(), dout.double().unsqueeze(1), y.double().view(T, k, H)
    dw, mag = (dd * yd).sum(2), (dd * yd).abs().sum(2)
    dy = (wd.unsqueeze(2) * dd).view(T * k, H)
    dz = torch.zeros(T, E, dtype=F64, device="cuda")
    dz.scatter_(1, ids.long(), wd * (dw - (wd * dw).sum(1, keepdim=True)))
    # a lane's chain of H / 64 products at most, then a tree over 64 lanes and 4 waves
    edw = (H / 64 + 12) * R.U32 * mag
    spread = (wd * (edw + (wd * edw).sum(1, keepdim=True)
                    + (k + 4) * R.U32 * (dw.abs() + (wd * dw.abs()).sum(1, keepdim=True))))
    edz = torch.zeros_like(dz).scatter_(1, ids.long(), spread)
    for extra in (None, add):
        r = ops.combine_backward(dout, y, ids, w, E, add=extra)
        _close(r["dy"], dy, dy.abs() * (R.half_step(dt) + 2 * R.U32), "dy")
        _close(r["dw"], dw, edw, "dw")
        want = dz if extra is None else dz + extra.double()
        _close(r["dlogits"], want, edz * 1.01 + 2 * R.U32 * (want.abs() + dz.abs()), "dlogits")


def test_combine_backward_against_differences():
    """The logits' gradient is that of sum(dout * combine(y, route(logits)))."""
    T, E, k, H = 6, 8, 3, 64
    logits = _rand(T, E, seed=1, dtype=F32)
    y, dout = _rand(T * k, H, seed=2, dtype=F32), _rand(T, H, seed=3, dtype=F32)
    ids, w = ops.route(logits, k)
    dz = ops.combine_backward(dout, y, ids, w, E)["dlogits"].double()

    def loss(z):
        p = torch.softmax(z.gather(1, ids.long()), 1)
        return ((p.unsqueeze(2) * y.double().view(T, k, H)).sum(1) * dout.double()).sum((1,))

    h = 1e-5
    for e in range(E):
        step = torch.zeros(T, E, dtype=F64, device="cuda")
        step[:, e] = h
        slope = (loss(logits.double() + step) - loss(logits.double() - step)) / (2 * h)
        # differences: h^2 times a third derivative of at most |dw| ~ 100; fp32 weights 1e-5
        assert (slope - dz[:, e]).abs().max() <= 1e-4


def test_combine_backward_bad_ids_and_in_place():
    T, E, k, H = 9, 5, 2, 72
    ids, w = ops.route(_rand(T, E, seed=1, dtype=F32), k)
    ids[2, 1], ids[4, 0] = E, -7
    gone = (ids < 0) | (ids >= E)
    y, dout = _rand(T * k, H, seed=2), _rand(T, H, seed=3)
    y.view(T, k, H)[gone] = float("nan")  # what a dropped pair's row holds is never read
    r = ops.combine_backward(dout, y, ids, w, E)
    assert not r["dy"].view(T, k, H)[gone].any() and not r["dw"][gone].any()
    assert all(torch.isfinite(t).all() for t in r.values())
    add = _rand(T, E, seed=4, dtype=F32)
    r2 = ops.combine_backward(dout, y, ids, w, E, add=add)
    lib, s = ops.lib(), torch.cuda.current_stream().cuda_stream
    dz, dy = add.clone(), y.clone()
    assert lib.qmoe_combine_backward(dout.data_ptr(), dy.data_ptr(), 0, ids.data_ptr(),
                                     w.data_ptr(), T, k, H, E, dz.data_ptr(), dy.data_ptr(), None,
                                     dz.data_ptr(), s) == 0
    assert torch.equal(dz, r2["dlogits"]) and torch.equal(dy, r2["dy"])

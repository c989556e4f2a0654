"""Far ends of the experts' bf16 products: factors whose product alone leaves fp32's
range, and operands behind the first 2 GiB."""
import pytest
import torch

import _block_ref as R
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


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


def _rows(n, cols, seed):
    """bf16 [n, cols] of a few values that repeat, made in place (the array is large)."""
    t = torch.empty(n, cols, dtype=BF, device="cuda")
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    part = torch.randn(1009, cols, generator=g, device="cuda").to(BF)
    for i in range(0, n, 1009):
        t[i:i + 1009] = part[:min(1009, n - i)]
    return t


def _sum_tol(n):
    return (n / 16 + 32) * R.U32 * 1.01


@pytest.mark.parametrize("pair_rows", [False, True])
def test_rows_of_a_behind_2_gib(pair_rows):
    """a of 2.9 GiB: the first, middle and last rows' products."""
    K, E, N = 4096, 3, 40
    rows = int(2.9 * (1 << 30)) // (2 * K) // 2 * 2
    k = 2
    T = rows // 2 if pair_rows else rows
    a = _rows(rows, K, 1)
    z = torch.arange(T, device="cuda", dtype=torch.int32)
    ids = torch.stack([z % 3, (z + 1) % 3], 1).contiguous()
    b = torch.randn(E, N, K, device="cuda").to(BF)
    al = ops.align(ids, E, 16)
    out = ops.grouped_matmul(a, b, al, k, pair_rows=pair_rows)
    dw = ops.grouped_wgrad(out, a, al, k, pair_rows=pair_rows)
    P = T * k
    flat = ids.reshape(-1).long()
    p = torch.cat([torch.arange(64), torch.arange(P // 2, P // 2 + 64), torch.arange(P - 64, P)])
    p = p.cuda()
    x = a[p if pair_rows else p // k].double()
    for e in range(E):
        of = flat[p] == e
        ref, mag = x[of] @ b[e].double().t(), x[of].abs() @ b[e].double().abs().t()
        assert ((out[p][of].double() - ref).abs() <= ref.abs() * R.BF16 + _sum_tol(K) * mag).all()
    # the weight gradient's sums over all rows of an expert, for a few columns of a
    cols = torch.tensor([0, 1, 2047, 4095], device="cuda")
    for e in range(E):
        of = (flat == e).nonzero().reshape(-1)
        ys = out[of].double()
        xs = a[:, cols][of if pair_rows else of // k].double()
        ref, mag = ys.t() @ xs, ys.abs().t() @ xs.abs()
        assert ((dw[e][:, cols].double() - ref).abs() <= _sum_tol(of.numel()) * mag).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T", [5, 700])
def test_a_matrix_of_b_behind_2_gib(T, trans):
    """One expert's matrix of 2.9 GiB: its last rows and columns."""
    K = 8192
    N = int(2.9 * (1 << 30)) // (2 * K) // 8 * 8
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    al = ops.align(ids, 1, 16)
    if trans:
        K, N = N, K
        b = _rows(K, N, 2).view(1, K, N)
        a = torch.randn(T, K, device="cuda").to(BF)
    else:
        b = _rows(N, K, 2).view(1, N, K)
        a = torch.randn(T, K, device="cuda").to(BF)
    out = ops.grouped_matmul(a, b, al, 1, trans=trans, out_dtype=F32)
    at = torch.cat([torch.arange(40), torch.arange(N // 2, N // 2 + 40), torch.arange(N - 40, N)])
    at = at.cuda()
    w = b[0][:, at].double() if trans else b[0][at].double().t()
    ref, mag = a.double() @ w, a.double().abs() @ w.abs()
    assert ((out[:, at].double() - ref).abs() <= _sum_tol(K) * mag).all()

"""bf16 expert products whose blocks take one tile after another: every tile that they
choose from, K of two, three and five blocks (the stages change roles from tile to tile
where their number is odd), each form, uneven rows and an expert without any.

Tolerances as in test_gpu_grouped.py."""
import pytest
import torch

import _block_ref as R
import _grouped_rule as rule
import test_gpu_grouped as G
from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def _one_each(counts, seed):
    """ids [P, 1] with these rows per expert."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    return flat[torch.randperm(flat.numel(), generator=g)].to(torch.int32).view(-1, 1).cuda()


def _two_each(counts):
    """ids [T, 2] with these rows per expert, a token's two distinct: the sorted list of
    experts against itself, half its length further on."""
    flat = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    T = flat.numel() // 2
    assert max(counts) <= T
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([flat[:T], flat[T:]], 1)[torch.randperm(T, generator=g)]
    assert (ids[:, 0] != ids[:, 1]).all()
    return ids.to(torch.int32).cuda()


@pytest.fixture(scope="module", autouse=True)
def _cus():
    if torch.cuda.get_device_properties(0).multi_processor_count != rule.CUS:
        pytest.skip("the sizes are for 256 CUs")


@pytest.mark.parametrize("K", [72, 136, 264])
@pytest.mark.parametrize("name,counts,N", rule.ROUNDS, ids=[r[0] for r in rule.ROUNDS])
def test_several_tiles_per_block(name, counts, N, K):
    print(f"rounds {name} N {N} K {K}", flush=True)
    E, P = len(counts), sum(counts)
    ids = _one_each(counts, K + N)
    al = ops.align(ids, E, 16)
    a = G._rand(P, K, seed=1, scale=2.0)
    nan = float("nan")
    tol = G._sum_tol(K) * 1.01

    b = G._rand(E, N, K, seed=2, scale=K ** -0.5)
    y, mag = G._plain(a, b, ids, True, False)
    for dt in (BF, F32):
        out = torch.full((P, N), nan, dtype=dt, device="cuda")
        ops.grouped_matmul(a, b, al, 1, pair_rows=True, out_dtype=dt, out=out)
        G._close(out, y, y.abs() * R.half_step(dt) + tol * mag, dt)
    # SiLU * mul, with and without gate and up
    g, u = y.chunk(2, 1)
    eg, eu = (tol * mag).chunk(2, 1)
    s = g * torch.sigmoid(g)
    err = 1.1 * u.abs() * eg + s.abs() * eu + 1.1 * eg * eu + 8 * R.U32 * (s * u).abs()
    gu = torch.full((P, N), nan, dtype=BF, device="cuda")
    h = ops.grouped_matmul(a, b, al, 1, act="silu_mul", gu=gu,
                           out=torch.full((P, N // 2), nan, dtype=BF, device="cuda"))
    G._close(h, s * u, (s * u).abs() * R.BF16 + err * 1.01, "silu")
    G._close(gu, y, y.abs() * R.BF16 + tol * mag, "gu")
    assert torch.equal(h, ops.grouped_matmul(a, b, al, 1, act="silu_mul"))
    h = ops.grouped_matmul(a, b, al, 1, act="silu_mul", out_dtype=F32)
    G._close(h, s * u, (s * u).abs() * R.U32 + err * 1.01, "silu fp32")
    del b, y, mag, g, u, eg, eu, s, err, gu, h, out

    b = G._rand(E, K, N, seed=3, scale=K ** -0.5)
    y, mag = G._plain(a, b, ids, True, True)
    for dt in (BF, F32):
        out = torch.full((P, N), nan, dtype=dt, device="cuda")
        ops.grouped_matmul(a, b, al, 1, pair_rows=True, trans=True, out_dtype=dt, out=out)
        G._close(out, y, y.abs() * R.half_step(dt) + tol * mag, ("turned", dt))
    gu = G._rand(P, 2 * N, seed=4, scale=3.0)
    g, u = gu.double().chunk(2, 1)
    f, s = G._silu_grad(g), g * torch.sigmoid(g)
    ref = torch.cat([y * u * f, y * s], 1)
    err = torch.cat([tol * mag * u.abs() * 1.1 + (y * u).abs() * 12 * 1.3 * R.U32,
                     tol * mag * s.abs() + 12 * R.U32 * (y * s).abs()], 1)
    for dt in (BF, F32):
        out = torch.full((P, 2 * N), nan, dtype=dt, device="cuda")
        ops.grouped_matmul(a, b, al, 1, pair_rows=True, trans=True, act="silu_mul_backward",
                           gu=gu, out_dtype=dt, out=out)
        G._close(out, ref, ref.abs() * R.half_step(dt) + err * 1.01, ("gradient", dt))


@pytest.mark.parametrize("name,counts,N", rule.ROUNDS, ids=[r[0] for r in rule.ROUNDS])
def test_rows_of_shared_tokens(name, counts, N):
    """Two pairs per token, so that a tile's rows of a are gathered out of order."""
    K = 136
    ids = _two_each(counts)
    E = len(counts)
    T = ids.shape[0]
    al = ops.align(ids, E, 16)
    a, b = G._rand(T, K, seed=5), G._rand(E, N, K, seed=6, scale=K ** -0.5)
    y, mag = G._plain(a, b, ids, False, False)
    got = ops.grouped_matmul(a, b, al, 2)
    G._close(got, y, y.abs() * R.BF16 + G._sum_tol(K) * 1.01 * mag, name)

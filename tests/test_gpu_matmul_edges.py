"""The fp8 products where K is split over blocks, and how exact they are."""
import pytest
import torch

from quantized_mixture_experts_moe_amd import ops
from test_gpu_block_ops import test_matmul as check_matmul

pytestmark = pytest.mark.gpu

# (rows, columns, K blocks, parts): 8 parts of 6, 8 parts with a short last one,
# K blocks that 7 parts of 7 take whole, a last part of one block, 4 and 2 parts
SPLITS = [(64, 256, 48, 8), (65, 129, 55, 8), (64, 256, 49, 7), (33, 64, 50, 8), (50, 190, 57, 8),
          (65, 129, 25, 4), (64, 2048, 33, 4), (40, 300, 13, 2), (64, 130, 11, 1)]


@pytest.mark.parametrize("b_block", [True, False])
@pytest.mark.parametrize("M,N,kb,parts", SPLITS)
def test_matmul_with_k_split(M, N, kb, parts, b_block):
    need = ops.fp8_matmul_workspace(M, N, 128 * kb)
    want = 4 * parts * M * N if parts > 1 else 0
    assert need == (want + 255) // 256 * 256
    check_matmul(M, N, 128 * kb, b_block)


def test_no_part_of_k_is_empty():
    """Whatever K is, the parts are as many as hold a K block each."""
    for kb in range(1, 200):
        need = ops.fp8_matmul_workspace(64, 64, 128 * kb)
        parts = max(1, need // (4 * 64 * 64))
        per = -(-kb // parts)
        assert (parts - 1) * per < kb, (kb, parts)

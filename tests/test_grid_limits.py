"""Products whose tiles no grid holds are refused before anything is launched."""
import ctypes
import os

import pytest
import torch

from quantized_mixture_experts_moe_amd import ops

pytestmark = [pytest.mark.skipif(not os.path.exists(ops.LIB_PATH),
                                 reason="libqmoe.so not built (run __graft_entry__.build())"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="addresses are not real ones")]
P = ctypes.c_void_p(0x10000)
INVALID_VALUE = 1  # hipErrorInvalidValue; without a GPU a launch has another error


def _refused(status):
    lib = ops.lib()
    return status == ops.QMOE_ERR_HIP and lib.qmoe_last_hip_error() == INVALID_VALUE


@pytest.mark.parametrize("rows", [20, 40, 100, 400])
def test_fp8_grouped_matmul(rows):
    """1024 experts of N columns and one K block; a hundredth of it would be launched."""
    def call(N):
        E = 1024
        return ops.lib().qmoe_fp8_grouped_matmul(P, P, 0, P, P, P, P, P, P, rows * E, 1, E, 16, N,
                                                 128, P, 0, None)
    assert _refused(call(1 << 24))
    assert not _refused(call(1 << 14))


def test_w4_matmul():
    """2^17 x 2^12 tiles of 128 x 128."""
    def call(M, N):
        return ops.lib().qmoe_w4_matmul(P, P, P, 0, 32, M, N, 32, 0, None, P, 0, None, 0, None)
    assert _refused(call(1 << 24, 1 << 19))
    assert not _refused(call(1 << 14, 1 << 14))

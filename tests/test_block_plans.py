"""What the operators around the experts choose by their sizes, as far as it
shows without a GPU."""
import os

import pytest

from quantized_mixture_experts_moe_amd import ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH),
                                reason="libqmoe.so not built (run __graft_entry__.build())")


def test_balance_of_many_tokens_takes_many_blocks():
    """Many tokens are shared by many blocks however few the experts are (the
    workspace is theirs); a few tokens are one block's, however many."""
    ws = ops.lib().qmoe_balance_workspace
    for T, E in ((4096, 8), (8192, 4), (1024, 32), (97, 1), (97, 1024), (1 << 20, 1)):
        assert ws(T, E) > 0, (T, E)
    for T, E in ((0, 8), (1, 1), (96, 1), (64, 512), (96, 1024)):
        assert ws(T, E) == 0, (T, E)


def test_the_operators_sources_contribute_kernels():
    """Every source of these operators is in the library, and the choices that
    they make by size find their kernels there."""
    import test_kernel_resources as K

    if not os.path.exists(K.READELF):
        pytest.skip("llvm-readelf is not available")
    names = " ".join(n for obj in K._code_objects(K.LIB) for n, _ in K._kernels(obj))
    for frag in ("fp8_quant_rows_kernel", "fp8_quant_tile_kernel", "fp8_matmul_rows_kernel",
                 "fp8_matmul_tile_kernel", "fp8_matmul_sum_kernel", "balance_small_kernel",
                 "balance_partial_kernel", "balance_finish_kernel", "balance_backward_kernel",
                 "pre_norm_kernel", "post_norm_kernel", "pre_norm_backward_kernel",
                 "post_norm_backward_kernel", "norm_colsum_kernel"):
        assert frag in names, frag

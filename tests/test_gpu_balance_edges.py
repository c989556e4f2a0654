"""The balance loss and its gradient on both sides of the choice between one
block and many, with few experts and many tokens."""
import pytest

from test_gpu_block_ops import test_balance as check_balance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", ["none", "some"])
@pytest.mark.parametrize("T,E,k", [(96, 4, 2), (97, 4, 2), (96, 1024, 16), (97, 1024, 16),
                                   (1024, 32, 4), (4096, 8, 2), (8192, 4, 2), (8195, 2, 2)])
def test_balance_on_both_sides_of_the_rule(T, E, k, masked):
    check_balance(T, E, k, masked)

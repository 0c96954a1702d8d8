"""Every form of the projection's product (a tile, whole or with K split) against
64 bits, forward and backward."""
import pytest

import test_gpu_proj
from proj_forms import FEW_SIZES, SIZES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("swap", [False, True], ids=["as listed", "K and N changed"])
@pytest.mark.parametrize("T,K,N,L,r", SIZES + FEW_SIZES + [(1001, 4096, 1024, 16, 16)])
def test_forms(T, K, N, L, r, swap):
    if swap:
        K, N = N, K
    test_gpu_proj.test_forward_and_backward(T, K, N, L, r, "mixed", True)

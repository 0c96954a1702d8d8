"""The dense operators' host side at the edges of what their contracts allow,
without a GPU."""
import ctypes

import pytest

import lora_moe_amd as lm

# addresses far apart that nothing ever reads: every call here is refused
BASE, STEP = 1 << 40, 1 << 36


@pytest.mark.parametrize("N,M,K", [(1, 9, 1024), (2, 9, 2048), (3, 10, 896), (1, 32, 1024), (2, 16, 1024),
                                   (5, 32, 1024), (64, 9, 2048)])
def test_slabs_of_a_few_bytes_are_asked_for(N, M, K):
    """A product that cannot do without a workspace never reports the 256
    bytes of one that can."""
    lib = lm.load_library()
    d = lm.moe_lora_w4(BASE, N, K, 128, 0)
    need = lib.moe_lora_w4_workspace_bytes(ctypes.byref(d), M)
    call = lambda ws, n: lib.moe_lora_w4_matmul(ctypes.byref(d), M, BASE + STEP, ws, n, BASE + 2 * STEP,  # noqa: E731
                                                None)
    assert call(None, 0) == lm.MOE_LORA_EWORKSPACE and call(BASE + 3 * STEP, 0) == lm.MOE_LORA_EWORKSPACE
    assert need >= 512

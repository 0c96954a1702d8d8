"""Operands without memory are refused where they might be left out, before
anything is written."""
import pytest
import torch

import lora_moe_amd as lm

pytestmark = pytest.mark.gpu


def none(*sizes, dtype=torch.float32):
    t = torch._efficientzerotensor(sizes, dtype=dtype, device="cuda")
    assert t.data_ptr() == 0 and t.is_contiguous()
    return t


def seven(*sizes, dtype=torch.bfloat16):
    return torch.full(sizes, 7, dtype=dtype, device="cuda")


def test_operands_without_memory_are_refused():
    T, H, k, E = 6, 64, 2, 5
    s = lm.make_sort_shape(T, H, E, k)
    row = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    y = seven(T, H)
    with pytest.raises(ValueError, match="weights has no memory"):
        lm.moe_lora_unsort(s, seven(T * k, H), row, y, weights=none(T, k))
    dw = seven(T, k, dtype=torch.float32)
    with pytest.raises(ValueError, match="drows has no memory"):
        lm.moe_lora_unsort_backward(s, seven(T, H), seven(T * k, H), row, drows=none(T * k, H, dtype=torch.bfloat16),
                                    dweights=dw)
    N, L, r = 32, 3, 8
    p = lm.make_proj_shape(T, H, N, L, r)
    q = seven(T, N)
    args = seven(T, H), torch.zeros(T, dtype=torch.int32, device="cuda"), seven(N, H), seven(L, r, H), seven(L, N, r)
    with pytest.raises(ValueError, match="scales has no memory"):
        lm.moe_lora_proj_forward(p, *args, lm.alloc_proj_workspace(p), q, scales=none(L))
    with pytest.raises(ValueError, match="workspace has no memory"):
        lm.moe_lora_proj_forward(p, *args, none(lm.moe_lora_proj_workspace_bytes(p), dtype=torch.uint8), q)
    f = lm.make_ffn_shape(T, H, 64)
    with pytest.raises(ValueError, match="gu has no memory"):
        lm.moe_lora_ffn_forward(f, seven(T, H), seven(128, H), seven(H, 64), lm.alloc_ffn_workspace(f), y,
                                gu=none(T, 128))
    torch.cuda.synchronize()
    assert bool((y == 7).all()) and bool((dw == 7).all()) and bool((q == 7).all())

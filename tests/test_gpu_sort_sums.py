"""The weights' gradient adds its products in few steps: each product is rounded
in its pair, its piece, its lane's sum and the lanes', not once for every product
before it."""
import math

import pytest
import torch

import lora_moe_amd as lm
from dense_common import HALF_F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1100, 40])
@pytest.mark.parametrize("dtype,H", [("float32", 2048), ("float32", 8192), ("bfloat16", 7168), ("float16", 4096)])
def test_small_products_are_not_lost_one_by_one(T, dtype, H):
    """Every lane meets a one first and half steps of it after that, which a
    chain of sums loses one by one."""
    t = getattr(torch, dtype)
    per = 16 // t.itemsize                       # values of a piece
    waves = 4 if T <= 1024 else 1
    pieces = math.ceil(H / per / (64 * waves))   # of a lane
    small = HALF_F32 if dtype != "float16" else 2.0 ** -12
    rows = torch.full((T, H), small, dtype=torch.float64)
    rows[:, 0:per * 64 * waves:per] = 1
    dy = torch.ones((T, H), dtype=t)
    if dtype == "float16":  # (2^-24 is none of its normal values)
        dy[:] = small
        dy[:, 0:per * 64 * waves:per] = 1
    s = lm.make_sort_shape(T, H, 4, 1, dtype)
    row = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).view(T, 1)
    dw = torch.empty((T, 1), device="cuda")
    lm.moe_lora_unsort_backward(s, dy.cuda(), rows.to(t).cuda(), row, dweights=dw)
    want = (rows.to(t).double() * dy.double()).sum(1, keepdim=True)
    steps = math.log2(per) + 1 + pieces + 6 + (waves - 1)
    assert float((dw.cpu().double() - want).abs().max()) <= steps * HALF_F32 * float(want[0])

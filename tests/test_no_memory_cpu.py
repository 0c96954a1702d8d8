"""An operand without memory is refused: its address is that of an operand that
was not given."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import lora_moe_amd as lm
from test_operands_cpu import CALLED, call


def fake(*sizes, dtype=torch.float32):
    with FakeTensorMode():
        return torch.empty(sizes, dtype=dtype, device="cuda")


def test_a_tensor_without_memory_is_not_passed():
    assert fake(4, 8).is_cuda and fake(4, 8).is_contiguous()
    assert call(("weights", fake(4, 8), (4, 8), "float32"), 9) is None and not CALLED
    assert call(5, ("workspace", fake(256, dtype=torch.uint8), None, "uint8"), None) is None and not CALLED
    # an empty one has none either, and is as good as any
    assert call(("weights", fake(0, 8), (0, 8), "float32"), 9) == 7 and CALLED[0][1:3] == (None, 9)


def test_it_is_said():
    with pytest.raises(ValueError, match="gu has no memory"):
        lm._address("gu", torch._efficientzerotensor((4, 8)))
    t = torch.zeros(4, 8)
    assert lm._address("gu", None) is None and lm._address("gu", t) == t.data_ptr()
    assert not lm._address("gu", t[:0])  # (or its storage's address)

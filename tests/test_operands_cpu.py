"""How the binding looks at its tensors before the library sees them, without
a GPU: what is refused, and that nothing is called then."""
import ctypes
import sys

import pytest
import torch

import lora_moe_amd as lm
from lora_moe_amd import _operands

CALLED = []
PROBE = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 17)(lambda *a: CALLED.append(a) or 7)
ADDRESS = ctypes.cast(PROBE, ctypes.c_void_p).value
SHAPE = lm.make_proj_shape(4, 64, 32, 2, 8)


def call(*args, device=0):
    CALLED.clear()
    return _operands.call(ADDRESS, SHAPE, args, device)


def test_a_call_passes_shape_numbers_and_null_pointers():
    assert call(5, None, 1 << 40) == 7
    shape, *rest = CALLED[0]
    assert shape == ctypes.addressof(SHAPE) and rest[:4] == [5, None, 1 << 40, None]


@pytest.mark.parametrize("tensor", [torch.zeros(4, 8), torch.zeros(8, 4).t(), torch.zeros(4, 8, requires_grad=True),
                                    torch.zeros(4, 8, device="meta"), torch.zeros(4, 8).to_sparse(), None, 3, "x"],
                         ids=["cpu", "strided", "leaf", "meta", "sparse", "none", "number", "text"])
def test_what_does_not_lie_on_the_device_is_not_passed(tensor):
    assert call(("x", tensor, (4, 8), "float32"), 9) is None and not CALLED
    assert call(("workspace", tensor, None, "uint8"), None, 9) is None and not CALLED


@pytest.mark.parametrize("args", [("x",), (("x", 3, (4, 8)),), (("x", 3, (4, 8), 5),), (("x", 3, [4, 8], "float32"),),
                                  (1.5,), (-1,), (1 << 64,), (None,) * 16])
def test_arguments_of_other_forms_are_refused(args):
    CALLED.clear()
    try:
        assert _operands.call(ADDRESS, SHAPE, args, 0) is None
    except (TypeError, OverflowError):
        pass
    assert not CALLED


def test_calls_of_other_forms_are_refused():
    CALLED.clear()
    for args in ((), (ADDRESS, SHAPE, ()), (ADDRESS, SHAPE, [], 0), (ADDRESS, 3, (), 0), ("f", SHAPE, (), 0)):
        with pytest.raises(TypeError):
            _operands.call(*args)
    assert not CALLED


def cpu(*sizes, dtype=torch.float32):
    return torch.zeros(sizes, dtype=dtype)


@pytest.mark.parametrize("shape", [lm.make_sort_shape(3, 64, 8, 2, "float32"), lm.make_proj_shape(3, 64, 8, 2, 8), None],
                         ids=["sort", "projection", "none"])
def test_a_structure_of_another_operator_is_refused(shape):
    """The sort's sizes have all the names that the router's gradient asks
    for, in a structure that ends long before the one it reads."""
    if isinstance(shape, lm.moe_lora_sort_shape):
        with pytest.raises(TypeError, match="shape: moe_lora_sort_shape, expected moe_lora_shape"):
            lm.moe_lora_route_backward(shape, cpu(3, 2, dtype=torch.int32), cpu(3, 2), cpu(3, 2), cpu(3, 8))
        return
    with pytest.raises((TypeError, AttributeError)):
        lm.moe_lora_unsort(shape, cpu(6, 64), cpu(3, 2, dtype=torch.int32), cpu(3, 64))
    with pytest.raises((TypeError, AttributeError)):
        lm.moe_lora_proj_forward(None, *[None] * 7)


def test_what_is_wrong_is_said():
    s, ids = lm.make_sort_shape(3, 64, 8, 2, "float32"), cpu(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="rows is required"):
        lm.moe_lora_unsort(s, None, ids, cpu(3, 64))
    with pytest.raises(ValueError, match="rows: dtype bfloat16, expected float32"):
        lm.moe_lora_unsort(s, cpu(6, 64, dtype=torch.bfloat16), ids, cpu(3, 64))
    with pytest.raises(ValueError, match=r"y: shape \(3, 63\), expected \(3, 64\)"):
        lm.moe_lora_unsort(s, cpu(6, 64), ids, cpu(3, 63))
    with pytest.raises(ValueError, match="rows must be contiguous"):
        lm.moe_lora_unsort(s, cpu(64, 6).t(), ids, cpu(3, 64))
    with pytest.raises(ValueError, match="operands must be device tensors"):
        lm.moe_lora_unsort(s, cpu(6, 64), ids, cpu(3, 64))


def test_without_the_module_it_says_how_to_build_it(monkeypatch):
    monkeypatch.setattr(lm, "_native", None)
    monkeypatch.delattr(lm, "_operands")
    monkeypatch.setitem(sys.modules, "lora_moe_amd._operands", None)
    with pytest.raises(RuntimeError, match="build it first"):
        lm.moe_lora_unsort(lm.make_sort_shape(3, 64, 8, 2), cpu(6, 64), cpu(3, 2), cpu(3, 64))

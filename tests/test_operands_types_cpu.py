"""The binding calls each library function through its own type, with as many
arguments as it takes."""
import ctypes

import pytest

import lora_moe_amd as lm
from lora_moe_amd import _operands

SHAPE = lm.make_proj_shape(4, 64, 32, 2, 8)


@pytest.mark.parametrize("name", sorted(_operands.kinds))
def test_a_function_gets_its_arguments(name):
    types = getattr(lm.load_library(), name).argtypes
    called = []
    probe = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, *types[1:])(lambda *a: called.append(a) or 3)
    address, kind = ctypes.cast(probe, ctypes.c_void_p).value, _operands.kinds[name]
    args = tuple((i + 1) << 34 for i in range(len(types) - 1))
    assert _operands.call(address, SHAPE, args, 0, kind) == 3
    assert called == [(ctypes.addressof(SHAPE), *args)]
    for other in (args[:-1], args + (5,), ()):
        with pytest.raises(TypeError):
            _operands.call(address, SHAPE, other, 0, kind)
    assert len(called) == 1


def test_every_operator_of_the_binding_has_a_kind():
    for kind in (-1, len(_operands.kinds) + 1, "moe_lora_sort", None):
        with pytest.raises(TypeError):
            _operands.call(1, SHAPE, (), 0, kind)
    assert sorted(_operands.kinds.values()) == list(range(len(_operands.kinds)))

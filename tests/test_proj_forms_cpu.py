"""The sizes that the GPU tests of the projection use meet every form of its
product, in both directions."""
import pytest

from proj_forms import FORMS, SIZES, form, sorted_forward
from test_gpu_proj_parts import CASES


@pytest.mark.parametrize("sizes", [SIZES, CASES], ids=["forms", "parts"])
def test_every_form_is_met(sizes):
    assert {form(T, K, N, r, False) for T, K, N, L, r in sizes if sorted_forward(T, N, L, r)} == FORMS
    # (a backward is always sorted; its sums run over N)
    assert {form(T, N, K, r, True) for T, K, N, L, r in sizes} == FORMS

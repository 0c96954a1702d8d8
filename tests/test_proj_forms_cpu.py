"""The sizes that the GPU tests of the projection use meet every form of its
product, in both directions."""
import pytest

import test_gpu_proj
from proj_forms import FEW_FORMS, FEW_SIZES, FORMS, SIZES, few_form, form, sorted_forward
from test_gpu_proj_parts import CASES


@pytest.mark.parametrize("sizes", [SIZES, CASES], ids=["forms", "parts"])
def test_every_form_is_met(sizes):
    assert {form(T, K, N, r, False) for T, K, N, L, r in sizes if sorted_forward(T, N, L, r)} == FORMS
    # (a backward is always sorted; its sums run over N)
    assert {form(T, N, K, r, True) for T, K, N, L, r in sizes} == FORMS


def test_every_form_of_decode_batches_is_met():
    sizes = [c[:5] for c in test_gpu_proj.CASES] + FEW_SIZES
    assert {few_form(*c) for c in sizes if not sorted_forward(c[0], *c[2:])} == FEW_FORMS

"""The sizes that the GPU tests of the projection use meet every form of its
product, in both directions."""
import pytest

import test_gpu_proj
from proj_forms import FEW_FORMS, FEW_SIZES, FORMS, SIZES, few_form, few_plan, form, sorted_forward
from test_gpu_proj_parts import CASES


@pytest.mark.parametrize("sizes", [SIZES, CASES], ids=["forms", "parts"])
def test_every_form_is_met(sizes):
    assert {form(T, K, N, r, False) for T, K, N, L, r in sizes if sorted_forward(T, N, L, r)} == FORMS
    # (a backward is always sorted; its sums run over N)
    assert {form(T, N, K, r, True) for T, K, N, L, r in sizes} == FORMS


def test_every_form_of_decode_batches_is_met():
    sizes = [c[:5] for c in test_gpu_proj.CASES] + FEW_SIZES
    assert {few_form(*c) for c in sizes if not sorted_forward(c[0], *c[2:])} == FEW_FORMS


def test_decode_batches_split_k_up_to_a_workgroup_per_cu():
    for T in (1, 8, 32, 33, 100, 256):
        for K in (264, 2880, 4096, 8192):
            for N in (264, 2880, 4088, 4096, 4104, 5120, 11008):
                tile, splits = few_plan(T, K, N, 8, 16)
                if tile not in ("32x64", "64x128"):
                    continue  # (the rule of the dense block's tiles)
                rows, cols = (32, 64) if tile == "32x64" else (64, 128)
                tiles = -(-T // rows) * -(-(N + 16 * min(8, T)) // cols)
                assert splits == 1 or splits * tiles <= 256, (T, K, N, tile, splits)

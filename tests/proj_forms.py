"""Sizes at which the projection's product takes each of its forms: a tile,
whole or with K split.  The rule is asked itself, so that a change of its
constants that loses a form is seen."""
import ctypes

import lora_moe_amd as lm

TILES = ("256x256", "128x128", "128x128 in two groups", "64x128", "32x64")
FORMS = {(t, split) for t in TILES[1:4] for split in (False, True)} | {("256x256", False)}
# of the product of decode batches, x [W; A]^T
FEW_FORMS = {(t, split) for t in TILES[1:] for split in (False, True)}

# T, K (summed over), N (outputs), L, r of sorted batches
SIZES = [(514, 136, 136, 3, 16), (520, 136, 72, 4, 128), (514, 8, 8, 4, 8), (2075, 752, 8, 3, 128),
         (2069, 8, 904, 5, 128), (1430, 3688, 8, 3, 128), (75, 2656, 3208, 31, 64), (2235, 288, 3824, 4, 128)]

# of batches without an order: forms that test_gpu_proj's sizes leave out
FEW_SIZES = [(257, 1632, 4880, 26, 64)]


def form(T, K, N, r, back):
    """The tile and whether K is split; back: of dx, whose sums run over N."""
    f = lm.load_library()._ZN7moelora14proj_gemm_planEiiiib
    f.argtypes, f.restype = [ctypes.c_int] * 4 + [ctypes.c_bool], ctypes.c_int
    plan = f(T, K, N, r, back)
    return TILES[plan // 32], plan % 32 > 1


def sorted_forward(T, N, L, r):
    """Whether a forward goes by the order (the rule of proj_few)."""
    f = lm.load_library()._ZN7moelora8proj_fewEiiii
    f.argtypes, f.restype = [ctypes.c_int] * 4, ctypes.c_bool
    return not f(T, N, L, r)


def few_plan(T, K, N, L, r):
    """The tile and the K splits of a batch without an order."""
    f = lm.load_library()._ZN7moelora14proj_both_planEiiiii
    f.argtypes, f.restype = [ctypes.c_int] * 5, ctypes.c_int
    plan = f(T, K, N, L, r)
    return TILES[plan // 32], plan % 32


def few_form(T, K, N, L, r):
    tile, splits = few_plan(T, K, N, L, r)
    return tile, splits > 1

"""The sort by expert, the way back and the router's gradient: host-side
checks; each refusal returns its code, or raises, without touching a GPU."""
import ctypes

import pytest
import torch

import lora_moe_amd as lm

OK, EINVAL, EALIGN, EWS, EUNSUP = (lm.MOE_LORA_OK, lm.MOE_LORA_EINVAL, lm.MOE_LORA_EALIGN, lm.MOE_LORA_EWORKSPACE,
                                   lm.MOE_LORA_EUNSUPPORTED)
BASE, STEP = 1 << 40, 1 << 38  # addresses far apart that nothing ever reads


def at(i, off=0):
    return BASE + i * STEP + off


@pytest.fixture(scope="module")
def lib():
    return lm.load_library()


ARGS = dict(
    moe_lora_sort=("topk_ids", "x", "ws", "n", "rows", "expert_off", "row_of_pair", "pair_of_row"),
    moe_lora_sort_backward=("drows", "row_of_pair", "dx"),
    moe_lora_unsort=("rows", "row_of_pair", "weights", "y"),
    moe_lora_unsort_backward=("dy", "rows", "row_of_pair", "weights", "drows", "dweights"),
    moe_lora_route_backward=("topk_ids", "weights", "dweights", "dlogits"))
OPTIONAL = {"pair_of_row", "weights"}


def call(lib, name, s, **over):
    a = {n: at(i) for i, n in enumerate(ARGS[name])}
    if "n" in a:
        a["n"] = 1 << 34
    a.update(over)
    return getattr(lib, name)(ctypes.byref(s) if s else None, *[a[n] for n in ARGS[name]], None)


@pytest.mark.parametrize("sizes,code", [
    ((-1, 64, 8, 2, 1), EINVAL), ((4, 0, 8, 2, 1), EINVAL), ((4, 64, 0, 2, 1), EINVAL), ((4, 64, 8, 0, 1), EINVAL),
    ((4, 64, 8, 9, 1), EINVAL), ((4, 64, 8, 2, 3), EINVAL), ((4, 64, 8, 2, -1), EINVAL), ((4, 60, 8, 2, 1), EALIGN),
    ((4, 60, 8, 2, 0), EALIGN), (((1 << 25) + 1, 8, 8, 1, 1), EUNSUP), ((4, (1 << 20) + 8, 8, 2, 1), EUNSUP),
    ((4, 64, 4097, 2, 1), EUNSUP), ((4, 64, 100, 65, 1), EUNSUP), ((1 << 25, 8, 64, 64, 1), EUNSUP)])
def test_sort_shapes(lib, sizes, code):
    s = lm.moe_lora_sort_shape(*sizes)
    for name in ARGS:
        if name != "moe_lora_route_backward":
            assert call(lib, name, s) == code, name
    assert lm.moe_lora_sort_workspace_bytes(s) == 0
    with pytest.raises(lm.MoeLoraError):
        lm.alloc_sort_workspace(s, device="cpu")


def test_sort_arguments(lib):
    s = lm.make_sort_shape(5, 64, 8, 3)
    for name, args in ARGS.items():
        shape = lm.make_shape(5, 64, 8, 8, 3, 1, 8) if name == "moe_lora_route_backward" else s
        assert call(lib, name, None) == EINVAL, name
        for n in args:
            if n in ("n", "ws") or n in OPTIONAL and name != "moe_lora_route_backward":
                continue
            if name == "moe_lora_unsort_backward" and n in ("drows", "dweights"):
                continue
            assert call(lib, name, shape, **{n: None}) == EINVAL, (name, n)
        for n in args:
            if n != "n":
                assert call(lib, name, shape, **{n: at(20, 4)}) == EALIGN, (name, n)
    need = lm.moe_lora_sort_workspace_bytes(s)
    assert call(lib, "moe_lora_sort", s, ws=None) == EWS
    assert call(lib, "moe_lora_sort", s, n=need - 1) == EWS
    assert call(lib, "moe_lora_unsort_backward", s, drows=None, dweights=None) == EINVAL
    # rows may be missing only where no dweights are wanted
    assert call(lib, "moe_lora_unsort_backward", s, rows=None) == EINVAL


def test_sort_overlaps(lib):
    """An output on an input or another output, by its first or last bytes."""
    s = lm.make_sort_shape(5, 64, 8, 3)
    last_x, last_pair = 5 * 64 * 2 - 16, 48  # 15 pairs: 60 bytes
    where = lambda name, n: ARGS[name].index(n)  # noqa: E731
    for name, out, other, off in (
            ("moe_lora_sort", "rows", "x", last_x), ("moe_lora_sort", "rows", "topk_ids", 0),
            ("moe_lora_sort", "row_of_pair", "topk_ids", last_pair), ("moe_lora_sort", "expert_off", "rows", 0),
            ("moe_lora_sort", "pair_of_row", "row_of_pair", last_pair), ("moe_lora_sort", "ws", "x", 0),
            ("moe_lora_sort", "ws", "expert_off", 32),
            ("moe_lora_sort_backward", "dx", "drows", 0), ("moe_lora_sort_backward", "dx", "row_of_pair", 48),
            ("moe_lora_unsort", "y", "rows", 3 * last_x), ("moe_lora_unsort", "y", "weights", 0),
            ("moe_lora_unsort_backward", "drows", "rows", 0), ("moe_lora_unsort_backward", "drows", "dy", last_x),
            ("moe_lora_unsort_backward", "dweights", "weights", 0),
            ("moe_lora_unsort_backward", "dweights", "drows", 16)):
        assert call(lib, name, s, **{out: at(where(name, other), off)}) == EINVAL, (name, out, other)
    r = lm.make_shape(5, 64, 8, 8, 3, 1, 8)
    for other in ("topk_ids", "weights", "dweights"):
        i = where("moe_lora_route_backward", other)
        assert call(lib, "moe_lora_route_backward", r, dlogits=at(i, 48)) == EINVAL, other


def test_route_backward_shapes(lib):
    for (T, E, k), code in (((-1, 8, 2), EINVAL), ((4, 0, 1), EINVAL), ((4, 8, 0), EINVAL), ((4, 8, 9), EINVAL),
                            ((4, 80, 65), EUNSUP), ((1 << 30, 256, 8), EUNSUP)):
        s = lm.moe_lora_shape(T, 8, 8, E, k, 1, 8, 0, 1.0)
        assert call(lib, "moe_lora_route_backward", s) == code, (T, E, k)


def test_no_tokens(lib):
    s = lm.make_sort_shape(0, 64, 8, 3)
    assert lm.moe_lora_sort_workspace_bytes(s) > 0
    for name in ("moe_lora_sort_backward", "moe_lora_unsort", "moe_lora_unsort_backward"):
        assert call(lib, name, s, **{n: None for n in ARGS[name]}) == OK, name
    r = lm.make_shape(0, 64, 8, 8, 3, 1, 8)
    assert call(lib, "moe_lora_route_backward", r, **{n: None for n in ARGS["moe_lora_route_backward"]}) == OK
    # the sort still writes expert_off
    assert call(lib, "moe_lora_sort", s, expert_off=None) == EINVAL


def test_sort_binding():
    with pytest.raises(ValueError, match="dtype"):
        lm.make_sort_shape(1, 8, 8, 1, dtype=torch.int32)
    assert lm.make_sort_shape(1, 8, 8, 1, torch.float16).dtype == lm.MOE_LORA_F16
    s = lm.make_sort_shape(2, 16, 4, 2)
    z = lambda *d, t=torch.bfloat16: torch.zeros(d, dtype=t)  # noqa: E731
    i = lambda *d: z(*d, t=torch.int32)  # noqa: E731
    ws = z(lm.moe_lora_sort_workspace_bytes(s), t=torch.uint8)
    good = dict(topk_ids=i(2, 2), x=z(2, 16), workspace=ws, rows=z(4, 16), expert_off=i(5), row_of_pair=i(2, 2))
    for over, text in ((dict(), "device tensors"), (dict(topk_ids=z(2, 2, t=torch.int64)), "dtype"),
                       (dict(x=z(2, 16, t=torch.float16)), "dtype"), (dict(rows=z(2, 16)), "shape"),
                       (dict(x=z(16, 2).t()), "contiguous"), (dict(x=None), "required"), (dict(rows=None), "required"),
                       (dict(workspace=ws[:4]), "workspace"), (dict(expert_off=i(4)), "shape"),
                       (dict(pair_of_row=i(2, 2)), "shape")):
        with pytest.raises(ValueError, match=text):
            lm.moe_lora_sort(s, **dict(good, **over))
    with pytest.raises(ValueError, match="shape"):
        lm.moe_lora_sort_backward(s, z(2, 16), i(2, 2), z(2, 16))
    with pytest.raises(ValueError, match="dtype"):
        lm.moe_lora_unsort(s, z(4, 16), i(2, 2), z(2, 16), weights=z(2, 2))
    with pytest.raises(ValueError, match="shape"):
        lm.moe_lora_unsort_backward(s, z(2, 16), z(4, 16), i(2, 2), dweights=z(4, t=torch.float32))
    with pytest.raises(ValueError, match="dtype"):
        f = z(2, 2, t=torch.float32)
        lm.moe_lora_route_backward(lm.make_shape(2, 8, 8, 4, 2, 1, 8), i(2, 2), f, f, z(2, 4))
    s.dtype = 7
    with pytest.raises(ValueError, match="dtype"):
        lm.moe_lora_sort_backward(s, z(4, 16), i(2, 2), z(2, 16))

"""Global gradient norm and clipping on the GPU against 64-bit forms."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def clip(lm, grads, max_norm, out=None, stream=None):
    norm = torch.full((1,), float("nan"), device="cuda")
    lm.moe_lora_clip_grads(lm.GradSet(grads, out) if out is not None else grads, max_norm, norm, stream=stream)
    return norm


def make(sizes, dtypes, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(dtypes[i % len(dtypes)]).cuda() for i, s in enumerate(sizes)]


def check(grads, outs, norm, max_norm):
    """fp64 sums: the norm is off by its fp32 rounding (and the fp64 sum's,
    below 2^-40); c is rounded to fp32 and the product once to fp32 and once
    to its type."""
    want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    assert abs(float(norm) - want) <= (2.0 ** -24 + 2.0 ** -40) * want
    c = min(1.0, max_norm / (want + 1e-6))
    for t, o in zip(grads, outs):
        ref = t.double() * c
        half = torch.finfo(t.dtype).eps / 2
        tiny = torch.finfo(t.dtype).smallest_normal * half  # half a step among subnormals
        bound = (half + 2 * 2.0 ** -24 + 2.0 ** -30) * ref.abs() + tiny * (1 + 2.0 ** -10)
        assert bool(((o.double() - ref).abs() <= bound).all()), (t.shape, t.dtype)


SETS = [[(1,)], [(7,), (0,), (16384,)], [(16385,), (3, 5), (100, 333), (1 << 18,)], [(1000003,)],
        [(i % 97 + 1, 3) for i in range(300)], [(0,), (0, 4)] + [(64,)] * 113 + [(0,)]]


@pytest.mark.parametrize("dtype", [0, 1, 2, None])
@pytest.mark.parametrize("sizes", range(len(SETS)))
def test_clip(sizes, dtype):
    import lora_moe_amd as lm
    grads = make(SETS[sizes], DTYPES if dtype is None else [DTYPES[dtype]], sizes)
    total = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    for max_norm in (0.37 * total, 2 * total, 0.0):
        outs = [torch.full_like(t, 3.0) for t in grads]
        n1 = clip(lm, grads, max_norm, outs)
        check(grads, outs, n1, max_norm)
        mine = [t.clone() for t in grads]
        n2 = clip(lm, mine, max_norm)  # in place
        assert torch.equal(n1, n2)
        for a, b in zip(mine, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_views(dtype, shift):
    """Gradients and outputs at odd offsets of larger buffers, not the same
    ones: what lies around them stays."""
    import lora_moe_amd as lm
    grads, outs, bufs = [], [], []
    g = torch.Generator().manual_seed(2)
    for n in (5, 1000, 16384 + 77, 40001):
        a = torch.full((n + 32,), 9.0, dtype=dtype, device="cuda")
        b = torch.full((n + 32,), 9.0, dtype=dtype, device="cuda")
        grads.append(a[shift:shift + n].copy_(torch.randn(n, generator=g)))
        off = 8 if n == 1000 else 2 * shift
        outs.append(b[off:off + n])
        bufs.append((b, off, n))
    norm = clip(lm, grads, 1.0, outs)
    check(grads, outs, norm, 1.0)
    for b, off, n in bufs:
        assert (b[:off] == 9).all() and (b[off + n:] == 9).all()


def test_norm_only():
    import lora_moe_amd as lm
    grads = make([(1000,), (33, 77)], DTYPES, 1)
    kept = [t.clone() for t in grads]
    check(grads, grads, clip(lm, grads, float("inf")), float("inf"))
    for a, b in zip(grads, kept):
        assert torch.equal(a, b)


def test_no_bound_leaves_gradients_that_are_not_finite():
    """max_norm = inf: every value goes on as it is, whatever the norm is."""
    import lora_moe_amd as lm
    for v in (float("inf"), float("nan")):
        grads = make([(1000,), (33, 77)], DTYPES, 1)
        grads[1][3, 5] = v
        outs = [torch.zeros_like(t) for t in grads]
        norm = clip(lm, grads, float("inf"), outs)
        assert not math.isfinite(float(norm))
        for a, b in zip(grads, outs):
            assert torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0))


def test_tensors_given_other_memory():
    """A set keeps the memory that it listed, and clips that."""
    import lora_moe_amd as lm
    g = torch.full((5000,), 2.0, device="cuda")
    old = g.detach()
    gs = lm.GradSet([g])
    g.data = torch.full((5000,), 3.0, device="cuda")
    norm = torch.empty(1, device="cuda")
    lm.moe_lora_clip_grads(gs, 1.0, norm)
    want = 2.0 * math.sqrt(5000)
    assert abs(float(norm) - want) <= 1e-6 * want
    assert torch.allclose(old, torch.full_like(old, 2.0 / want), rtol=1e-5) and (g == 3.0).all()


def test_no_tensors():
    import lora_moe_amd as lm
    assert float(clip(lm, [], 1.0)) == 0.0
    e = [torch.empty(0, device="cuda"), torch.empty((0, 3), dtype=torch.bfloat16, device="cuda")]
    assert float(clip(lm, e, 1.0)) == 0.0


def test_large_and_small_values():
    """Squares past fp32's range and below it."""
    import lora_moe_amd as lm
    for v in (1e30, 1e-30):
        grads = [torch.full((1000,), v, device="cuda"), torch.full((50,), -v, device="cuda")]
        outs = [torch.empty_like(t) for t in grads]
        norm = clip(lm, grads, 0.5 * v, outs)
        want = v * math.sqrt(1050)
        assert abs(float(norm) - want) <= 1e-6 * want
        if v > 1:
            c = 0.5 * v / want
            assert torch.allclose(outs[0], grads[0] * c, rtol=1e-6)


def test_values_that_are_not_finite():
    import lora_moe_amd as lm
    grads = make([(100,), (20,)], [torch.float32], 1)
    grads[0][7] = float("inf")
    outs = [torch.empty_like(t) for t in grads]
    assert float(clip(lm, grads, 1.0, outs)) == float("inf")
    assert torch.isnan(outs[0][7]) and not outs[0][:7].any() and not outs[1].any()
    grads[0][7] = float("nan")
    assert math.isnan(float(clip(lm, grads, 1.0, outs)))
    assert torch.isnan(outs[0]).all() and torch.isnan(outs[1]).all()


def test_same_bits_and_graph_replays():
    import lora_moe_amd as lm
    grads = make([(50000,), (3, 999)] + [(70,)] * 200, DTYPES, 3)
    outs = [torch.empty_like(t) for t in grads]
    gs = lm.GradSet(grads, outs)
    norm = torch.empty(1, device="cuda")
    lm.moe_lora_clip_grads(gs, 2.0, norm)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        lm.moe_lora_clip_grads(gs, 2.0, norm, stream=s)
    for rep in range(3):
        for t, n in zip(grads, make([t.shape for t in grads], DTYPES, 10 + rep)):
            t.copy_(n)
        e_out = [torch.empty_like(t) for t in grads]
        e_norm = clip(lm, grads, 2.0, e_out)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, e_norm)
        for a, b in zip(outs, e_out):
            assert torch.equal(a, b), rep


def test_another_stream():
    import lora_moe_amd as lm
    grads = make([(5000,), (70, 3)], DTYPES, 4)
    want = clip(lm, [t.clone() for t in grads], 1.0)
    norm = torch.empty(1, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lm.moe_lora_clip_grads(grads, 1.0, norm, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(norm, want)

"""Tokens sorted by expert and back, their gradients and the router's, against
64 bits.

Bounds: a sum of n fp32 terms t_i is off by at most (n + 1) 2^-24 sum |t_i|
whatever its order (each product and each addition rounds by half a step, and
a later one meets what an earlier one left), then a result is rounded to its
type by half a step: 2^-8 (bf16), 2^-11 (fp16, and 2^-25 absolute among its
subnormals), 2^-24 (fp32)."""
import pytest
import torch

import lora_moe_amd as lm

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
GUARD = 64


def near(got, want, bound, dtype, what):
    bound = bound + HALF[dtype] * (want.abs() + bound) + (2.0 ** -25 if dtype is torch.float16 else 1e-40)
    err = (got.double().cpu() - want).abs()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    worst = float((err / bound).max()) if err.numel() else 0.0
    print(f"[{what}] worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, (what, worst)


def guarded(shape, dtype, fill):
    """A tensor with GUARD elements of its fill behind it, and a check."""
    n = 1
    for d in shape:
        n *= d
    flat = torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")
    return flat[:n].view(shape), lambda: bool((flat[n:] == fill).all())


def order64(ids, E):
    """expert_off, row_of_pair, pair_of_row by the definition, one pair after
    the other."""
    flat = ids.reshape(-1).tolist()
    counts = [0] * (E + 1)
    for e in flat:
        if 0 <= e < E:
            counts[e + 1] += 1
    off = [0] * (E + 1)
    for e in range(E):
        off[e + 1] = off[e] + counts[e + 1]
    at, row, pair = list(off), [], {}
    for p, e in enumerate(flat):
        if 0 <= e < E:
            row.append(at[e])
            pair[at[e]] = p
            at[e] += 1
        else:
            row.append(-1)
    return torch.tensor(off), torch.tensor(row, dtype=torch.int64).reshape(ids.shape), pair


def ids_of(kind, T, E, k, g):
    if kind == "one":      # every pair the same expert: the same index many times
        return torch.full((T, k), E - 1, dtype=torch.int32)
    if kind == "dropped":  # a third of the pairs without an expert, both kinds of bad id
        ids = torch.randint(0, E, (T, k), generator=g)
        bad = torch.rand((T, k), generator=g)
        return torch.where(bad < 0.2, -1, torch.where(bad < 0.33, E + 3, ids)).int()
    if kind == "none":
        return torch.full((T, k), -1, dtype=torch.int32)
    return torch.rand((T, E), generator=g).topk(k, dim=1)[1].int()


CASES = [  # T, H, E, k, dtype, ids
    (1, 8, 1, 1, torch.bfloat16, "router"), (1, 4096, 8, 2, torch.float16, "router"),
    (16, 2880, 32, 4, torch.float32, "router"), (7, 72, 5, 5, torch.bfloat16, "dropped"),
    (33, 264, 3, 3, torch.float16, "one"), (65, 2048, 4096, 6, torch.bfloat16, "router"),
    (129, 64, 300, 64, torch.float32, "dropped"), (1001, 512, 128, 8, torch.bfloat16, "dropped"),
    (1025, 80, 17, 8, torch.float16, "router"), (1024, 64, 8, 8, torch.bfloat16, "one"),
    (1030, 64, 8, 8, torch.float32, "one"), (2999, 136, 256, 3, torch.bfloat16, "dropped"),
    (9001, 24, 7, 7, torch.bfloat16, "router"), (20000, 16, 4096, 1, torch.float16, "dropped"),
    (40, 96, 9, 2, torch.bfloat16, "none"), (5000, 96, 9, 2, torch.bfloat16, "none")]


@pytest.mark.parametrize("T,H,E,k,dtype,kind", CASES)
def test_sort_and_back(T, H, E, k, dtype, kind):
    g = torch.Generator().manual_seed(T * 7 + E)
    ids = ids_of(kind, T, E, k, g)
    x, d, dy, dxs = ((torch.randn(s, generator=g) * m).to(dtype) for s, m in (
        ((T, H), 1.0), ((T * k, H), 1.0), ((T, H), 0.1), ((T * k, H), 0.1)))
    w = torch.rand((T, k), generator=g)
    off, row, pair = order64(ids, E)
    used = int(off[-1])
    shape = lm.make_sort_shape(T, H, E, k, dtype)
    ws = lm.alloc_sort_workspace(shape)
    rows, ok0 = guarded((T * k, H), dtype, 7.0)
    offs, ok1 = guarded((E + 1,), torch.int32, -9)
    rop, ok2 = guarded((T, k), torch.int32, -9)
    por, ok3 = guarded((T * k,), torch.int32, -9)
    dev = [t.cuda() for t in (ids, x, d, dy, dxs, w)]
    lm.moe_lora_sort(shape, dev[0], dev[1], ws, rows, offs, rop, por)
    assert torch.equal(offs.cpu().long(), off) and torch.equal(rop.cpu().long(), row)
    want_pair = torch.full((T * k,), -9, dtype=torch.int32)
    for r, p in pair.items():
        want_pair[r] = p
    assert torch.equal(por.cpu(), want_pair)
    want = torch.full((T * k, H), 7.0, dtype=dtype)
    want[:used] = x[want_pair[:used].long() // k]
    assert torch.equal(rows.cpu(), want), "rows"
    # the order alone gives the same
    o2, r2 = torch.empty_like(offs), torch.empty_like(rop)
    lm.moe_lora_sort(shape, dev[0], None, ws, None, o2, r2)
    assert torch.equal(o2, offs) and torch.equal(r2, rop)

    has = (row >= 0).double()
    at = row.clamp(min=0)
    for weights, what in ((w, "weights"), (None, "ones")):
        y, ok4 = guarded((T, H), dtype, 7.0)
        lm.moe_lora_unsort(shape, dev[2], rop, y, weights=None if weights is None else dev[5])
        w64 = has * (1.0 if weights is None else weights.double())
        terms = d.double()[at] * w64[:, :, None]
        near(y, terms.sum(1), (k + 1) * HALF[torch.float32] * terms.abs().sum(1), dtype, f"y, {what}")
        drows, ok5 = guarded((T * k, H), dtype, 7.0)
        dw, ok6 = guarded((T, k), torch.float32, 7.0)
        lm.moe_lora_unsort_backward(shape, dev[3], dev[2], rop, drows, weights=None if weights is None else dev[5],
                                    dweights=dw)
        want = torch.full((T * k, H), 7.0, dtype=torch.float64)
        for j in range(k):
            m = row[:, j] >= 0
            want[row[m, j]] = dy.double()[m] * w64[m, j][:, None]
        near(drows, want, HALF[torch.float32] * want.abs(), dtype, f"drows, {what}")
        prod = d.double()[at] * dy.double()[:, None, :] * has[:, :, None]
        near(dw, prod.sum(2), (H + 1) * HALF[torch.float32] * prod.abs().sum(2), torch.float32, f"dweights, {what}")
        assert bool((dw.cpu()[row < 0] == 0).all())
        assert ok4() and ok5() and ok6()
        # each alone
        only, only_w = torch.full_like(drows, 7.0), torch.empty_like(dw)
        lm.moe_lora_unsort_backward(shape, dev[3], None, rop, only, weights=None if weights is None else dev[5])
        lm.moe_lora_unsort_backward(shape, dev[3], dev[2], rop, weights=None if weights is None else dev[5],
                                    dweights=only_w)
        assert torch.equal(only, drows) and torch.equal(only_w, dw)
    dx, ok7 = guarded((T, H), dtype, 7.0)
    lm.moe_lora_sort_backward(shape, dev[4], rop, dx)
    terms = dxs.double()[at] * has[:, :, None]
    near(dx, terms.sum(1), (k + 1) * HALF[torch.float32] * terms.abs().sum(1), dtype, "dx")
    assert ok0() and ok1() and ok2() and ok3() and ok7()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 4), (5, 6, 3), (3, 256, 8), (1000, 128, 8), (777, 33, 7),
                                   (64, 500, 64), (8193, 64, 6), (2, 7168, 8)])
def test_route_backward(T, E, k):
    """Against the softmax's Jacobian, and against differences of the router's
    own weights."""
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn((T, E), generator=g)
    shape = lm.make_shape(T, 8, 8, E, k, 1, 8)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    lm.moe_lora_route(shape, logits.cuda(), ids, w)
    dw = torch.randn((T, k), generator=g)
    out, ok = guarded((T, E), torch.float32, 7.0)
    lm.moe_lora_route_backward(shape, ids, w, dw.cuda(), out)
    i64, w64, dw64 = ids.cpu().long(), w.double().cpu(), dw.double()
    s = (w64 * dw64).sum(1, keepdim=True)
    # the sum is off by (k + 1) half steps of its terms, then a difference and a product
    e = w64 * ((k + 1) * (w64 * dw64).abs().sum(1, keepdim=True) + 2 * (dw64.abs() + s.abs())) * HALF[torch.float32]
    want = torch.zeros((T, E), dtype=torch.float64).scatter_(1, i64, w64 * (dw64 - s))
    bound = torch.zeros((T, E), dtype=torch.float64).scatter_(1, i64, e * 1.01)
    near(out, want, bound, torch.float32, "dlogits")
    assert bool((out.cpu()[bound == 0] == 0).all()) and ok()
    # differences in 64 bits, the choice held: f(logits) = sum_j dw_j softmax(chosen)_j
    chosen = logits.double().gather(1, i64)
    f = lambda v: (torch.softmax(v, 1) * dw64).sum(1)  # noqa: E731
    h = 1e-5
    for j in range(min(k, 4)):
        step = torch.zeros_like(chosen)
        step[:, j] = h
        diff = (f(chosen + step) - f(chosen - step)) / (2 * h)
        got = out.double().cpu().gather(1, i64[:, j:j + 1])[:, 0]
        # the router's weights are fp32 (1e-6 of the softmax), differences of third order h^2
        assert float((diff - got).abs().max()) <= 1e-5 * float(dw64.abs().max()), j


def test_route_backward_slots():
    """Slots without an expert take no part, whatever their numbers; a repeated
    id gets the sum; large values stay finite."""
    ids = torch.tensor([[2, -1, 5], [-1, -1, -1], [3, 3, 0], [9, 1, -7]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.75, 0, 0.25], [0, 0, 0], [0.5, 0.25, 0.25], [float("nan"), 1.0, float("inf")]], device="cuda")
    nan = float("nan")
    dw = torch.tensor([[1.0, nan, 3.0], [nan, 1.0, float("inf")], [4.0, 2.0, 0.0], [nan, 3e38, nan]], device="cuda")
    for E in (6, 8):  # one and four logits a thread
        shape = lm.make_shape(4, 8, 8, E, 3, 1, 8)
        out = torch.full((4, E), 7.0, device="cuda")
        lm.moe_lora_route_backward(shape, ids, w, dw, out)
        want = torch.zeros((4, E))
        want[0, 2], want[0, 5] = 0.75 * (1 - 1.5), 0.25 * (3 - 1.5)
        want[2, 3], want[2, 0] = 0.5 * (4 - 2.5) + 0.25 * (2 - 2.5), 0.25 * (0 - 2.5)
        assert torch.equal(out.cpu(), want)


def test_bad_rows_are_dropped():
    """Indexes outside the rows are pairs without one, not addresses."""
    shape = lm.make_sort_shape(3, 16, 4, 2)
    big = 2 ** 31 - 1
    rop = torch.tensor([[0, 6], [-1, big], [-big, 5]], dtype=torch.int32, device="cuda")
    rows = torch.arange(96, dtype=torch.bfloat16, device="cuda").view(6, 16)
    y = torch.empty((3, 16), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_unsort(shape, rows, rop, y)
    assert torch.equal(y, torch.stack((rows[0], torch.zeros_like(rows[0]), rows[5])))
    drows = torch.full_like(rows, 3.0)
    dw = torch.empty((3, 2), device="cuda")
    lm.moe_lora_unsort_backward(shape, y, rows, rop, drows, dweights=dw)
    want = torch.full_like(rows, 3.0)
    want[0], want[5] = y[0], y[2]
    assert torch.equal(drows, want)
    assert dw.cpu()[0, 1] == 0 and dw.cpu()[1].tolist() == [0, 0] and dw.cpu()[2, 0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_values_that_are_not_finite(dtype):
    """Rows are copied bit for bit; sums meet infinities and NaN by the formula,
    and another token's never."""
    T, H, E, k = 6, 24, 4, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H), generator=g).to(dtype)
    x[1, 3], x[2, 5], x[3] = float("inf"), float("nan"), torch.finfo(dtype).min
    ids = ids_of("router", T, E, k, g)
    shape = lm.make_sort_shape(T, H, E, k, dtype)
    rows = torch.empty((T * k, H), dtype=dtype, device="cuda")
    offs = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rop = torch.empty((T, k), dtype=torch.int32, device="cuda")
    lm.moe_lora_sort(shape, ids.cuda(), x.cuda(), lm.alloc_sort_workspace(shape), rows, offs, rop)
    row = rop.cpu().long()
    for t in range(T):
        for j in range(k):
            a, b = rows[row[t, j]].cpu().view(torch.uint8), x[t].contiguous().view(torch.uint8)
            assert torch.equal(a, b)
    y = torch.empty((T, H), dtype=dtype, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    lm.moe_lora_unsort(shape, rows, rop, y, weights=w)
    # halves of one value twice: the value itself
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=77.0), torch.nan_to_num(x, nan=77.0))


def test_offsets_past_32_bits():
    """Rows of more than 2^31 elements (and 4 GiB): the last rows are right."""
    T, H, k = 1100, 1 << 20, 2
    shape = lm.make_sort_shape(T, H, 4, k)
    ids = torch.tensor([0, 3], dtype=torch.int32, device="cuda").repeat(T, 1)
    x = torch.randint(-4, 5, (T, 1), device="cuda").to(torch.bfloat16).repeat(1, H)
    x[:, -1] = torch.arange(T, device="cuda") % 251
    rows = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    offs = torch.empty(5, dtype=torch.int32, device="cuda")
    rop = torch.empty((T, k), dtype=torch.int32, device="cuda")
    lm.moe_lora_sort(shape, ids, x, lm.alloc_sort_workspace(shape), rows, offs, rop)
    assert rows.numel() > 2 ** 31
    assert torch.equal(rows[:T], x) and torch.equal(rows[T:], x)
    y = torch.empty_like(x)
    lm.moe_lora_unsort(shape, rows, rop, y)
    assert torch.equal(y, x + x)
    drows = torch.empty_like(rows)
    dw = torch.empty((T, k), device="cuda")
    lm.moe_lora_unsort_backward(shape, x, rows, rop, drows, dweights=dw)
    assert torch.equal(drows, rows)
    want = x[:, 0].double() ** 2 * (H - 1) + x[:, -1].double() ** 2
    assert float((dw.double() - want[:, None]).abs().max()) <= float(want.max()) * 2.0 ** -23


def test_streams_and_replays():
    """On another stream than the current one, and captured and replayed with
    new inputs between: each equals the eager result bit for bit."""
    T, H, E, k = 700, 256, 32, 4
    shape = lm.make_sort_shape(T, H, E, k)
    route = lm.make_shape(T, H, 8, E, k, 1, 8)
    g = torch.Generator(device="cuda").manual_seed(5)

    def inputs():
        logits = torch.randn((T, E), generator=g, device="cuda")
        v, ids = logits.topk(k, 1)
        r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        return [ids.int(), torch.softmax(v, 1), r(T, H), r(T * k, H), r(T, H), r(T * k, H)]

    def outputs():
        e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        return [e(T * k, H), e(E + 1, t=torch.int32), e(T, k, t=torch.int32), e(T, H), e(T * k, H),
                e(T, k, t=torch.float32), e(T, H), e(T, E, t=torch.float32)]

    def step(a, o, ws, stream=None):
        ids, w, x, d, dy, dxs = a
        lm.moe_lora_sort(shape, ids, x, ws, o[0], o[1], o[2], stream=stream)
        lm.moe_lora_unsort(shape, d, o[2], o[3], weights=w, stream=stream)
        lm.moe_lora_unsort_backward(shape, dy, d, o[2], o[4], weights=w, dweights=o[5], stream=stream)
        lm.moe_lora_sort_backward(shape, dxs, o[2], o[6], stream=stream)
        lm.moe_lora_route_backward(route, ids, w, o[5], o[7], stream=stream)

    sets = [inputs() for _ in range(3)]
    want = []
    for a in sets:
        o = outputs()
        step(a, o, lm.alloc_sort_workspace(shape))
        want.append(o)
    side, o = torch.cuda.Stream(), outputs()
    ws = lm.alloc_sort_workspace(shape)
    side.wait_stream(torch.cuda.current_stream())
    step(sets[1], o, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(o, want[1]))
    live, o = [t.clone() for t in sets[0]], outputs()
    step(live, o, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(live, o, ws)
    for i in (1, 2, 0, 2):
        for t, s in zip(live, sets[i]):
            t.copy_(s)
        for t in o:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(o, want[i])), i
        step(sets[(i + 1) % 3], outputs(), lm.alloc_sort_workspace(shape))

"""The shared projection with the adapters of many requests, forward and
backward, against 64 bits within bounds from the roundings (proj_common.py)."""
import pytest
import torch

import lora_moe_amd as lm
from dense_common import within
from proj_common import backward64, forward64, inputs

pytestmark = pytest.mark.gpu

GUARD = 64


def guarded(shape, dtype=torch.bfloat16):
    n = 1
    for d in shape:
        n *= d
    flat = torch.full((n + GUARD,), 7.0, dtype=dtype, device="cuda")
    return flat[:n].view(shape), lambda: bool((flat[n:] == 7.0).all())


def workspace(shape, backward=True):
    """A workspace of the least size with a guard behind it, full of NaN."""
    n = lm.moe_lora_proj_workspace_bytes(shape, backward)
    flat = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    return flat[:n], lambda: bool((flat[n:] == 255).all())


CASES = [  # T, K, N, L, r, ids, scales
    (1, 8, 8, 1, 8, "each", True), (1, 4096, 4096, 8, 16, "each", True), (1, 264, 136, 3, 128, "none", True),
    (2, 136, 2880, 5, 24, "mixed", False), (5, 1000, 72, 2, 40, "one", True), (8, 512, 520, 64, 8, "each", True),
    (9, 72, 1032, 4, 72, "mixed", True), (16, 2880, 512, 16, 32, "each", False), (17, 200, 200, 40, 16, "mixed", True),
    (32, 4096, 1000, 16, 64, "each", True), (32, 640, 96, 100, 128, "mixed", True),
    (33, 136, 136, 3, 8, "mixed", True), (33, 8, 8, 2, 16, "each", True), (64, 1000, 520, 64, 16, "each", False),
    (130, 256, 512, 4, 8, "runs", True), (201, 2880, 640, 32, 16, "each", True), (257, 72, 2880, 7, 128, "mixed", True),
    (300, 264, 264, 300, 24, "each", True), (513, 512, 136, 9, 72, "runs", True), (700, 200, 1032, 2, 40, "none", True),
    (1030, 520, 392, 5, 64, "mixed", False), (1100, 136, 264, 3, 32, "one", True), (2100, 264, 640, 16, 16, "runs", True),
    (4500, 136, 264, 6, 16, "runs", True), (4200, 264, 136, 4, 96, "mixed", True),
    (201, 264, 200, 32, 16, "each", True), (90, 1000, 520, 40, 128, "mixed", True), (33, 136, 2880, 500, 8, "each", True),
    (1300, 264, 4104, 9, 72, "each", True), (600, 2880, 2880, 16, 32, "runs", True),
    # every tile: small ones whole and with K split, deep ones, large ones
    (2100, 2056, 2064, 3, 16, "each", True), (1400, 2056, 2064, 5, 24, "runs", True),
    (1832, 16, 2216, 2, 16, "runs", True), (2423, 1368, 8, 3, 128, "mixed", True), (194, 2760, 6904, 53, 64, "each", True),
    (260, 1032, 4104, 6, 8, "each", True), (500, 136, 6000, 40, 8, "mixed", True),
    (8192, 1032, 4096, 3, 16, "runs", True), (8192, 1032, 4096, 37, 40, "mixed", False)]


@pytest.mark.parametrize("T,K,N,L,r,ids,scales", CASES)
def test_forward_and_backward(T, K, N, L, r, ids, scales):
    x, W, A, B, dy, i, s = inputs(T, K, N, L, r, T + r, ids, scales)
    scale = 0.75
    shape = lm.make_proj_shape(T, K, N, L, r, scale)
    d = [t.cuda() for t in (x, W, A, B, dy, i)]
    ds = None if s is None else s.cuda()
    y, ok_y = guarded((T, N))
    z, ok_z = guarded((T, r), torch.float32)
    ws, ok_ws = workspace(shape, False)
    lm.moe_lora_proj_forward(shape, d[0], d[5], d[1], d[2], d[3], ws, y, z=z, scales=ds)
    assert ok_ws() and ok_y() and ok_z()
    # (the 64-bit forms on the GPU, the largest case would take half a minute)
    f = [t.double() for t in d[:5]]
    (z64, e_z), (y64, e_y) = forward64(*f[:4], d[5], ds, scale)
    within(z, z64.cpu(), e_z.cpu(), "z")
    within(y, y64.cpu(), e_y.cpu(), "y")
    assert bool((z.cpu()[(i < 0) | (i >= L)] == 0).all())
    y2 = torch.empty_like(y)  # without z
    ws, ok_ws = workspace(shape)
    lm.moe_lora_proj_forward(shape, d[0], d[5], d[1], d[2], d[3], ws, y2, scales=ds)
    assert torch.equal(y, y2)
    dx, ok_x = guarded((T, K))
    dA, ok_a = guarded((L, r, K))
    dB, ok_b = guarded((L, N, r))
    lm.moe_lora_proj_backward(shape, d[4], d[0], d[5], z, d[1], d[2], d[3], ws, dx=dx, dA=dA, dB=dB, scales=ds)
    assert ok_ws() and ok_x() and ok_a() and ok_b()
    want = backward64(f[4], f[0], z.double(), *f[1:4], d[5], ds, scale)
    for n, t in (("dx", dx), ("dA", dA), ("dB", dB)):
        within(t, want[n][0].cpu(), want[n][1].cpu(), n)
    # each alone, and none of them touches another's memory
    for n, t in (("dx", dx), ("dA", dA), ("dB", dB)):
        one = torch.empty_like(t)
        lm.moe_lora_proj_backward(shape, d[4], d[0], d[5], z, d[1], d[2], d[3], ws, scales=ds, **{n: one})
        assert torch.equal(one, t), n


def test_whole_numbers_and_differences():
    """On small whole numbers everything is exact, so that the loss dy . y of
    the kernel's own forward changes by exactly its gradients' products with a
    change of x, A or B (of one factor of z, in which y is linear)."""
    T, K, N, L, r = 70, 40, 24, 3, 8
    g = torch.Generator().manual_seed(3)
    few = lambda shape, p: ((torch.rand(shape, generator=g) < p).float()  # noqa: E731
                            * torch.randint(-1, 2, shape, generator=g)).bfloat16()
    x, W, A, B, dy = few((T, K), 0.3), few((N, K), 0.3), few((L, r, K), 0.2), few((L, N, r), 0.3), few((T, N), 0.3)
    ids = torch.randint(-1, L, (T,), generator=g).int()
    shape = lm.make_proj_shape(T, K, N, L, r, 2.0)
    ws = lm.alloc_proj_workspace(shape)
    z = torch.empty((T, r), device="cuda")

    def loss(x, A, B):
        y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        lm.moe_lora_proj_forward(shape, x.cuda(), ids.cuda(), W.cuda(), A.cuda(), B.cuda(), ws, y, z=z)
        assert float(y.abs().max()) <= 256
        return float((y.cpu().double() * dy.double()).sum())

    base = loss(x, A, B)
    out = {n: torch.empty_like(t, device="cuda") for n, t in (("dx", x), ("dA", A), ("dB", B))}
    lm.moe_lora_proj_backward(shape, dy.cuda(), x.cuda(), ids.cuda(), z, W.cuda(), A.cuda(), B.cuda(), ws, **out)
    for n, t in (("dx", x), ("dA", A), ("dB", B)):
        assert float(out[n].abs().max()) <= 256
        for k in range(4):
            e = few(t.shape, 0.02)
            moved = dict(x=x, A=A, B=B)
            moved[n[1:]] = (t + e).bfloat16()
            assert loss(**moved) - base == float((out[n].cpu().double() * e.double()).sum()), (n, k)


@pytest.mark.parametrize("T,L", [(7, 4), (20, 4), (90, 4), (600, 4), (90, 10), (600, 10), (1500, 30)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_broken_adapter_stays_with_its_tokens(T, L, bad):
    """Weights that are not finite reach the rows of their own adapter, by the
    formula, and no others."""
    K, N, r = 136, 264, 16
    x, W, A, B, dy, i, _ = inputs(T, K, N, L, r, 5, "each", False)
    shape = lm.make_proj_shape(T, K, N, L, r)
    ws = lm.alloc_proj_workspace(shape)

    def run(A, B):
        y, dx, dA, dB = (torch.empty_like(t, device="cuda") for t in (dy, x, A, B))
        z = torch.empty((T, r), device="cuda")
        a = [t.cuda() for t in (x, i, W, A, B, dy)]
        lm.moe_lora_proj_forward(shape, a[0], a[1], a[2], a[3], a[4], ws, y, z=z)
        lm.moe_lora_proj_backward(shape, a[5], a[0], a[1], z, a[2], a[3], a[4], ws, dx=dx, dA=dA, dB=dB)
        return [t.cpu() for t in (y, dx, dA, dB)]

    want = run(A, B)
    A2, B2 = A.clone(), B.clone()
    B2[2, 5, 3] = bad       # one output of adapter 2
    A2[1, 4, 9] = bad       # one rank of adapter 1
    y, dx, dA, dB = run(A2, B2)
    of = lambda l: i == l  # noqa: E731
    clean = ~(of(1) | of(2))
    assert torch.equal(y[clean], want[0][clean]) and torch.equal(dx[clean], want[1][clean])
    other = torch.ones(N, dtype=torch.bool)
    other[5] = False
    assert torch.equal(y[of(2)][:, other], want[0][of(2)][:, other])
    assert not torch.isfinite(y[of(2)][:, 5]).any() and not torch.isfinite(y[of(1)]).any()
    if bad == bad:  # the sign of an infinity is that of its term
        z = x.double() @ A[2, 3].double()
        sure = of(2) & (z.abs() > 1e-3)
        assert torch.equal(torch.sign(y[sure][:, 5].float()), torch.sign(z[sure] * bad).float())
    assert not torch.isfinite(dx[of(2)]).any() and not torch.isfinite(dx[of(1)][:, 9]).any()
    inner = torch.ones(K, dtype=torch.bool)
    inner[9] = False
    assert torch.equal(dx[of(1)][:, inner], want[1][of(1)][:, inner])
    for l in (0, 3, L - 1):
        assert torch.equal(dA[l], want[2][l]) and torch.equal(dB[l], want[3][l])


def test_tokens_that_are_not_finite():
    """A row of x with an infinity or NaN gives rows of y that are not finite
    and leaves the others alone, whatever tile they share."""
    for T in (6, 32, 150):
        x, W, A, B, dy, i, s = inputs(T, 72, 136, 3, 24, 9, "each")
        shape = lm.make_proj_shape(T, 72, 136, 3, 24)
        ws = lm.alloc_proj_workspace(shape)
        a = [t.cuda() for t in (i, W, A, B)]
        y, y2 = torch.empty_like(dy, device="cuda"), torch.empty_like(dy, device="cuda")
        lm.moe_lora_proj_forward(shape, x.cuda(), *a, ws, y, scales=s.cuda())
        x[1, 3], x[4, 70] = float("inf"), float("nan")
        lm.moe_lora_proj_forward(shape, x.cuda(), *a, ws, y2, scales=s.cuda())
        fine = torch.ones(T, dtype=torch.bool)
        fine[1] = fine[4] = False
        assert torch.equal(y.cpu()[fine], y2.cpu()[fine])
        assert not torch.isfinite(y2.cpu()[~fine]).any()


def test_large_values_of_z():
    """z between bf16's range and fp32's, and beyond 2^16 steps of a pair's
    remainder, stays finite."""
    for T in (4, 40):
        K, N, r = 8, 16, 8
        x = torch.zeros((T, K), dtype=torch.bfloat16)
        x[:, 0] = 2.0 ** 100
        x[:, 1] = 1.5
        W = torch.zeros((N, K), dtype=torch.bfloat16)
        A = torch.zeros((1, r, K), dtype=torch.bfloat16)
        A[0, 0, 0] = 2.0 ** 27 * 1.9921875      # z_0 = 2^127 * 1.9921875: bf16's largest
        A[0, 0, 1] = 2.0 ** 118                 # and a half step more
        B = torch.zeros((1, N, r), dtype=torch.bfloat16)
        B[0, :, 0] = 2.0 ** -100
        shape = lm.make_proj_shape(T, K, N, 1, r)
        y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        lm.moe_lora_proj_forward(shape, x.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"), W.cuda(), A.cuda(),
                                 B.cuda(), lm.alloc_proj_workspace(shape), y)
        z = 2.0 ** 127 * 1.9921875 + 1.5 * 2.0 ** 118
        want = torch.full((T, N), z * 2.0 ** -100, dtype=torch.float64).bfloat16()
        assert torch.equal(y.cpu(), want), T


def exact_small(shape, g, p=0.05):
    return ((torch.rand(shape, generator=g, device="cuda") < p)
            * torch.randint(-2, 3, shape, generator=g, device="cuda")).bfloat16()


def test_offsets_up_to_the_limit():
    """x of nearly 2^31 bytes, every token another request's; whole numbers."""
    T, K, N, L, r = 1 << 17, 8184, 8, 5, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    cols = torch.randint(0, K, (T, 4), generator=g, device="cuda")
    x.scatter_(1, cols, torch.ones((T, 4), dtype=torch.bfloat16, device="cuda"))
    W, A, B = exact_small((N, K), g), exact_small((L, r, K), g), exact_small((L, N, r), g, 0.3)
    ids = torch.randint(-1, L, (T,), generator=g, device="cuda").int()
    shape = lm.make_proj_shape(T, K, N, L, r)
    assert x.numel() * 2 > 2 ** 31 - 2 ** 22
    ws = lm.alloc_proj_workspace(shape)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((T, r), device="cuda")
    lm.moe_lora_proj_forward(shape, x, ids, W, A, B, ws, y, z=z)
    # by the few ones of each row
    has, l = (ids >= 0)[:, None].float(), ids.clamp(min=0).long()
    hit = torch.zeros_like(cols, dtype=torch.bool)
    for j in range(4):  # a column drawn twice counts once
        hit[:, j] = ~(cols[:, :j] == cols[:, j:j + 1]).any(1)
    z64 = sum(A.float()[l, :, cols[:, j]] * hit[:, j:j + 1] for j in range(4)) * has
    y64 = sum(W.float()[:, cols[:, j]].T * hit[:, j:j + 1] for j in range(4))
    y64 = y64 + (B.float()[l] * z64[:, None, :]).sum(2)
    assert torch.equal(z, z64) and torch.equal(y.float(), y64)
    dy = exact_small((T, N), g, 0.3)
    dx = torch.empty_like(x)
    dA = torch.empty_like(A)
    lm.moe_lora_proj_backward(shape, dy, x, ids, z, W, A, B, ws, dx=dx, dA=dA)
    u = (B.float()[l] * dy.float()[:, :, None]).sum(1) * has
    for a in (0, T // 2, T - 1000):
        rows = slice(a, a + 1000)
        want = dy[rows].float() @ W.float() + (u[rows][:, :, None] * A.float()[l[rows]]).sum(1)
        assert torch.equal(dx[rows].float(), want), a
    for a in range(L):
        at = ids == a
        want = torch.zeros((r, K), device="cuda")
        for j in range(4):
            want.index_add_(1, cols[at, j], (u[at] * hit[at, j:j + 1]).T)
        assert torch.equal(dA[a], want.bfloat16()), a


def test_adapters_up_to_the_limit():
    """Stacks of nearly 2^31 bytes, 2047 adapters."""
    L, r, K, N = 2047, 128, 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(4)
    A = torch.zeros((L, r, K), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((L, N, r), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    number = torch.arange(L, device="cuda")
    A[number, number % r, (number * 7) % K] = 1.0
    B[number, (number * 5) % N, number % r] = (number % 200 + 1).bfloat16()
    for T in (24, 3000):
        ids = torch.randint(0, L, (T,), generator=g, device="cuda").int()
        ids[0], ids[-1] = L - 1, 0
        x = torch.randint(1, 4, (T, K), generator=g, device="cuda").bfloat16()
        shape = lm.make_proj_shape(T, K, N, L, r)
        y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        z = torch.empty((T, r), device="cuda")
        ws = lm.alloc_proj_workspace(shape, False)
        lm.moe_lora_proj_forward(shape, x, ids, W, A, B, ws, y, z=z)
        i = ids.long()
        v = x[torch.arange(T, device="cuda"), (i * 7) % K].float()
        want = torch.zeros((T, N), device="cuda")
        want[torch.arange(T, device="cuda"), (i * 5) % N] = v * (i % 200 + 1)
        assert torch.equal(y, want.bfloat16())


def test_no_tokens():
    shape = lm.make_proj_shape(0, 64, 32, 3, 8)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ids, z = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 8), device="cuda")
    W, A, B = e(32, 64), e(3, 8, 64), e(3, 32, 8)
    ws = lm.alloc_proj_workspace(shape)
    lm.moe_lora_proj_forward(shape, e(0, 64), ids, W, A, B, ws, e(0, 32))
    dA, dB = torch.full_like(A, 3.0), torch.full_like(B, 3.0)
    lm.moe_lora_proj_backward(shape, e(0, 32), e(0, 64), ids, z, W, A, B, ws, dx=e(0, 64), dA=dA, dB=dB)
    assert bool((dA == 0).all()) and bool((dB == 0).all())


@pytest.mark.parametrize("T", [12, 400])
def test_streams_and_replays(T):
    K, N, L, r = 264, 392, 6, 24
    shape = lm.make_proj_shape(T, K, N, L, r)
    sets = [[t.cuda() for t in inputs(T, K, N, L, r, 40 + n, "each")] for n in range(3)]

    def outputs():
        e = lambda s, t=torch.bfloat16: torch.full(s, 9.0, dtype=t, device="cuda")  # noqa: E731
        return [e((T, N)), e((T, r), torch.float32), e((T, K)), e((L, r, K)), e((L, N, r))]

    def step(a, o, ws, stream=None):
        x, W, A, B, dy, ids, s = a
        lm.moe_lora_proj_forward(shape, x, ids, W, A, B, ws, o[0], z=o[1], scales=s, stream=stream)
        lm.moe_lora_proj_backward(shape, dy, x, ids, o[1], W, A, B, ws, dx=o[2], dA=o[3], dB=o[4], scales=s,
                                  stream=stream)

    want = []
    for a in sets:
        o = outputs()
        step(a, o, lm.alloc_proj_workspace(shape))
        want.append(o)
    side, o, ws = torch.cuda.Stream(), outputs(), lm.alloc_proj_workspace(shape)
    side.wait_stream(torch.cuda.current_stream())
    step(sets[1], o, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(o, want[1]))
    y = lm.lora_projection(sets[2][0], sets[2][5], *sets[2][1:4], scales=sets[2][6], stream=side)
    side.synchronize()
    assert torch.equal(y, want[2][0])
    live, o = [t.clone() for t in sets[0]], outputs()
    step(live, o, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(live, o, ws)
    for n in (1, 2, 0, 2):
        for t, s in zip(live, sets[n]):
            t.copy_(s)
        for t in o:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(o, want[n])), n
        step(sets[(n + 1) % 3], outputs(), lm.alloc_proj_workspace(shape))

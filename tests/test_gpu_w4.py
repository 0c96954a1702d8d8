"""4-bit products and the gated block on 4-bit weights on the GPU, against
64-bit forms within bounds from the roundings."""
import pytest
import torch

from dense_common import HALF_BF16, HALF_F32, LIP, act64, w4_bounds, w4_inputs, w4_values, within

pytestmark = pytest.mark.gpu


def rows(M, K, seed):
    return torch.randn((M, K), generator=torch.Generator().manual_seed(seed)).bfloat16()


def pack(lm, parts, group):
    q, s, z = (None if t is None else t.cuda() for t in parts)
    return lm.moe_lora_w4_pack(q, s, z, group=group)


def product(lm, x, w, stream=None):
    y = torch.full((x.shape[0], w.N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_w4_matmul(x, w, y, stream=stream)
    return y


# rows around every row tile; N odd, one and around 16; K around a chunk, with
# a last group that is short
SIZES = [(1, 16, 128), (1, 1, 8), (1, 4096, 4096), (2, 17, 136), (3, 1000, 2880), (4, 33, 72), (5, 250, 1000),
         (8, 515, 512), (9, 64, 3080), (15, 100, 256), (16, 48, 640), (17, 31, 1032), (31, 129, 264),
         (33, 300, 392), (48, 77, 2056), (63, 16, 520), (64, 1008, 1024), (65, 40, 136), (100, 200, 328),
         (130, 57, 776)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, group, zeros):
    import lora_moe_amd as lm
    parts = w4_inputs(N, K, group, zeros, 31 * N + K)
    x = rows(M, K, M)
    w = pack(lm, parts, group)
    xd = x.cuda()
    y = product(lm, xd, w)
    want, _, bound = w4_bounds(x.double(), *w4_values(*parts, group))
    within(y, want, bound, f"M={M} N={N} K={K} group={group} zeros={zeros}")
    assert torch.equal(product(lm, xd, w), y)


def test_rows_are_their_own():
    """A row's result has the same bits alone and among others, whatever the
    others hold."""
    import lora_moe_amd as lm
    N, K, group = 130, 1000, 64
    w = pack(lm, w4_inputs(N, K, group, True, 5), group)
    for M in (2, 7, 16, 20, 50, 64, 70):
        x = rows(M, K, 9).cuda()
        y = product(lm, x, w)
        x[M // 2] = float("nan")
        x[0, 3] = float("inf")
        yb = product(lm, x, w)
        for m in range(1, M):
            if m != M // 2:
                assert torch.equal(yb[m], y[m]), (M, m)
        assert not torch.isfinite(yb[M // 2]).any() and not torch.isfinite(yb[0]).any()


def test_integers_are_exact():
    """x of ones and unit scales: y is the sum of q - z, exact below 256."""
    import lora_moe_amd as lm
    N, K, group = 37, 96, 32
    q, s, z = w4_inputs(N, K, group, True, 3)
    s = torch.ones_like(s)
    w = pack(lm, (q, s, z), group)
    v, _ = w4_values(q, s, z, group)
    for k in range(0, K, 7):
        x = torch.zeros((3, K), dtype=torch.bfloat16)
        x[0, k] = 1
        x[1, k] = -2
        y = product(lm, x.cuda(), w).double().cpu()
        assert torch.equal(y[0], v[:, k]) and torch.equal(y[1], -2 * v[:, k]) and not y[2].any(), k


def test_zero_points_above_fifteen_count_as_fifteen():
    import lora_moe_amd as lm
    q, s, z = w4_inputs(20, 64, 32, True, 4)
    z[3] = 200
    a = product(lm, rows(2, 64, 1).cuda(), pack(lm, (q, s, z), 32))
    z[3] = 15
    b = product(lm, rows(2, 64, 1).cuda(), pack(lm, (q, s, z), 32))
    assert torch.equal(a, b)


def test_memory_around_is_left_alone():
    import lora_moe_amd as lm
    for M, N, K, group in ((1, 37, 200, 128), (5, 50, 136, 32), (21, 17, 72, 64), (64, 90, 264, 32)):
        parts = w4_inputs(N, K, group, True, 12)
        w = pack(lm, parts, group)
        x = rows(M, K, 2).cuda()
        xb = torch.full((M * K + 512,), float("nan"), dtype=torch.bfloat16, device="cuda")
        xv = xb[256:256 + M * K].view(M, K)
        xv.copy_(x)
        yb = torch.full((M * N + 65,), 7.0, dtype=torch.bfloat16, device="cuda")
        yv = yb[33:33 + M * N].view(M, N)  # y needs no alignment beyond its elements'
        lm.moe_lora_w4_matmul(xv, w, yv)
        assert torch.equal(yv, product(lm, x, w))
        assert (yb[:33] == 7).all() and (yb[33 + M * N:] == 7).all()


BLOCKS = [(1, 64, 72, 32), (2, 264, 136, 128), (5, 512, 1000, 64), (16, 136, 520, 32), (17, 104, 200, 128),
          (40, 328, 264, 64), (64, 256, 512, 128), (70, 72, 88, 32)]


def block(lm, x, ws3, act, stream=None):
    wsp = lm.alloc_w4_ffn_workspace(x.shape[0], ws3[0].N)
    y = torch.full((x.shape[0], ws3[2].N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_w4_ffn_forward(x, *ws3, wsp, y, act=act, stream=stream)
    return y


@pytest.mark.parametrize("act,zeros", [("silu", False), ("gelu", True)])
@pytest.mark.parametrize("M,H,I,group", BLOCKS)
def test_block(M, H, I, group, act, zeros):
    import lora_moe_amd as lm
    parts = [w4_inputs(I, H, group, zeros, 1), w4_inputs(I, H, group, zeros, 2), w4_inputs(H, I, group, zeros, 3)]
    x = rows(M, H, 40 + M)
    y = block(lm, x.cuda(), [pack(lm, p, group) for p in parts], act)
    vals = [w4_values(*p, group) for p in parts]
    g, e_g, _ = w4_bounds(x.double(), *vals[0])
    u, e_u, _ = w4_bounds(x.double(), *vals[1])
    a, _ = act64(g, act)
    h = a * u
    e_a = LIP * e_g + 64 * HALF_F32 * (a.abs() + g.abs())
    e_h = e_a * u.abs() + (a.abs() + e_a) * e_u
    e_h = e_h + HALF_BF16 * (h.abs() + e_h)
    want, e, _ = w4_bounds(h, *vals[2])
    e = e * 1.01 + e_h @ vals[2][0].abs().T + (I + 8) * HALF_F32 * (e_h @ vals[2][1].T)
    within(y, want, e + HALF_BF16 * (want.abs() + e), f"M={M} H={H} I={I} group={group} {act}")


def test_graph_replays_and_streams():
    """Captured once, replayed on new rows; and two products at once."""
    import lora_moe_amd as lm
    ws3 = [pack(lm, w4_inputs(n, k, 64, False, s), 64) for n, k, s in ((200, 136, 1), (200, 136, 2), (136, 200, 3))]
    x = rows(4, 136, 0).cuda()
    wsp = lm.alloc_w4_ffn_workspace(4, 200)
    y = torch.empty((4, 136), dtype=torch.bfloat16, device="cuda")
    block(lm, x, ws3, "silu")
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        lm.moe_lora_w4_ffn_forward(x, *ws3, wsp, y, stream=s)
    for rep in range(3):
        x2 = rows(4, 136, 70 + rep).cuda()
        want = block(lm, x2, ws3, "silu")
        x.copy_(x2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), rep
    xs = [rows(m, 136, m).cuda() for m in (3, 33)]
    alone = [product(lm, t, ws3[0]) for t in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [product(lm, t, ws3[0]) for t in xs]
    torch.cuda.synchronize()
    for t, y2, st in zip(xs, got, streams):
        y2.fill_(0)
        st.wait_stream(torch.cuda.current_stream())
        lm.moe_lora_w4_matmul(t, ws3[0], y2, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a, b)

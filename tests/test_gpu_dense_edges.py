"""Calls of the dense operators at the edges of what their contracts allow."""
import ctypes
import math

import pytest
import torch

from dense_common import ffn_inputs, w4_bounds, w4_inputs, w4_values, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 8, 9, 16])
@pytest.mark.parametrize("sign", [1, -1])
def test_pairs_between_the_ranges(T, sign):
    """h, dg or du within fp32's range and past bf16's (2^128 - 2^116): as a
    sum of two bf16 each is finite, and so is what takes half of it, 2^127 -
    2^115, which rounds to 2^127."""
    import lora_moe_amd as lm
    H, I = 64, 64
    z = lambda *d: torch.zeros(d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, W_gu, W_down = z(T, H), z(2 * I, H), z(H, I)
    x[:, 0], x[:, 1] = 2.0 ** 62, 2.0 ** 52
    W_gu[5, 0] = 4  # g = 2^64
    W_gu[I + 5, 0], W_gu[I + 5, 1] = 4 * sign, -sign  # u = 2^64 - 2^52
    W_down[:, 5] = 0.5
    shape = lm.make_ffn_shape(T, H, I)
    ws = lm.alloc_ffn_workspace(shape)
    y, gu = z(T, H), torch.empty((T, 2 * I), device="cuda")
    for kept in (gu, None):
        lm.moe_lora_ffn_forward(shape, x, W_gu, W_down, ws, y, gu=kept)
        assert (y == sign * 2.0 ** 127).all(), y
    assert (gu[:, 5] == 2.0 ** 64).all() and (gu[:, I + 5] == sign * (2.0 ** 64 - 2.0 ** 52)).all()
    # dh = 2^64: dg = du = h in size; a token each (or token 0's alone) in the weights' gradients
    dy, dx, dW_gu, dW_down = z(T, H), z(T, H), z(2 * I, H), z(H, I)
    dy[0, 3] = 2.0 ** 65
    x = z(T, H)
    x[0, 7] = 0.5
    gu = torch.zeros((T, 2 * I), device="cuda")
    gu[:, 5], gu[:, I + 5] = 2.0 ** 64 - 2.0 ** 52, sign * (2.0 ** 64 - 2.0 ** 52)
    W_gu = z(2 * I, H)
    W_gu[5, 11] = W_gu[I + 5, 12] = 0.5
    lm.moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, ws, dx=dx, dW_gu=dW_gu)
    assert dx[0, 11] == sign * 2.0 ** 127 and dx[0, 12] == 2.0 ** 127, dx[0, 11:13]
    assert dW_gu[5, 7] == sign * 2.0 ** 127 and dW_gu[I + 5, 7] == 2.0 ** 127
    # h = g u = 2^128 - 2^116 beside a dy of one half
    gu[:, 5] = 2.0 ** 64
    dy[0, 3] = 0.5
    lm.moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, ws, dW_down=dW_down)
    assert dW_down[3, 5] == sign * 2.0 ** 127, dW_down[3, 5]


@pytest.mark.parametrize("H,I", [(72, 40), (2056, 5512)])
def test_no_tokens_with_an_address_for_dx(H, I):
    """T = 0 from C with all three gradients: the weights' are zeros, dx is
    empty and what lies at its address stays."""
    import lora_moe_amd as lm
    lib = lm.load_library()
    W_gu, W_down = (torch.full(s, 2.0, dtype=torch.bfloat16, device="cuda") for s in ((2 * I, H), (H, I)))
    dW_gu, dW_down = torch.full_like(W_gu, 3.0), torch.full_like(W_down, 3.0)
    there = torch.full((256,), 7.0, dtype=torch.bfloat16, device="cuda")
    shape = lm.make_ffn_shape(0, H, I)
    stream = torch.cuda.current_stream().cuda_stream
    for dx in (there.data_ptr(), None):
        rc = lib.moe_lora_ffn_backward(ctypes.byref(shape), None, None, None, W_gu.data_ptr(), W_down.data_ptr(),
                                       None, 0, dx, dW_gu.data_ptr(), dW_down.data_ptr(), stream)
        assert rc == lm.MOE_LORA_OK
        assert not dW_gu.any() and not dW_down.any() and (there == 7).all()
        dW_gu.fill_(3.0)
        dW_down.fill_(3.0)


@pytest.mark.parametrize("N,M,K", [(1, 9, 1024), (2, 9, 2048), (3, 10, 896), (1, 32, 1024), (2, 16, 1024),
                                   (5, 32, 1024)])
def test_few_outputs_without_a_workspace(N, M, K):
    """K split over the grid with slabs of a few bytes: the binding finds
    their memory."""
    import lora_moe_amd as lm
    parts = w4_inputs(N, K, 128, False, N + K)
    w = lm.moe_lora_w4_pack(parts[0].cuda(), parts[1].cuda(), group=128)
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).bfloat16()
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_w4_matmul(x.cuda(), w, y)
    want, _, bound = w4_bounds(x.double(), *w4_values(*parts, 128))
    within(y, want, bound, f"M={M} N={N} K={K}")


def pool_of(t):
    """The stream whose memory the allocator gave to t."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("by_handle", [False, True])
def test_buffers_are_memory_of_the_stream_that_writes_them(by_handle):
    """On another stream, given as an object or by its handle, results are
    that stream's memory, and right; on the current one they are its own."""
    import lora_moe_amd as lm
    x, W_gu, W_down, _ = (t.cuda() for t in ffn_inputs(40, 136, 200, 3))
    parts = [t.cuda() for t in w4_inputs(300, 2048, 64, True, 4)]
    rows = torch.randn((20, 2048), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = []
    for s in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        st = s.cuda_stream if s and by_handle else s
        y, w = lm.gated_ffn(x, W_gu, W_down, stream=st), lm.moe_lora_w4_pack(*parts, group=64, stream=st)
        here = torch.cuda.current_stream().cuda_stream
        for t in (y, w.packed):
            assert pool_of(t) == (s.cuda_stream if s else here)
        out = torch.zeros((20, 300), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        lm.moe_lora_w4_matmul(rows, w, out, stream=st)
        torch.cuda.synchronize()
        want.append((y, w.packed, out))
        assert torch.cuda.current_stream().cuda_stream == here
    for a, b in zip(*want):
        assert torch.equal(a, b)


def test_a_set_of_gradients_on_several_streams():
    """One set, clipped on the current stream, under others and captured:
    the same norm everywhere, and each stream's partial sums in memory of its
    own, which replays use after the eager calls' has changed."""
    import lora_moe_amd as lm
    gen = torch.Generator().manual_seed(6)
    grads = [torch.randn(n, generator=gen).cuda() for n in (5000, 33, 70000)]
    outs = [torch.empty_like(t) for t in grads]
    gs = lm.GradSet(grads, outs)
    norms = torch.zeros((4, 1), device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    lm.moe_lora_clip_grads(gs, 2.0, norms[0])
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        lm.moe_lora_clip_grads(gs, 2.0, norms[1])
    torch.cuda.synchronize()
    lm.moe_lora_clip_grads(gs, 2.0, norms[2], stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    handles = [torch.cuda.current_stream().cuda_stream] + [s.cuda_stream for s in streams]
    assert [pool_of(gs._workspace(h)) for h in handles] == handles
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lm.moe_lora_clip_grads(gs, 2.0, norms[3])
    for rep in range(3):
        lm.moe_lora_clip_grads([grads[1].clone()], 2.0, torch.empty(1, device="cuda"))
        norms[3].zero_()
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(n, norms[0]) for n in norms), (rep, norms)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_norm_of_a_few_elements(dtype):
    """Sums of squares are fp64: the norm of the 1 to 9 elements around one
    16-byte piece is off by its own rounding to fp32 alone, draw for draw."""
    import lora_moe_amd as lm
    gen = torch.Generator().manual_seed(11)
    n = 4 if dtype is torch.float32 else 8
    for size in (1, n - 1, n, n + 1):
        host = torch.randn((250, size), generator=gen).to(dtype)
        norms = torch.empty((250, 1), device="cuda")
        for t, norm in zip(host.cuda(), norms):
            lm.moe_lora_clip_grads([t.clone()], math.inf, norm)
        want = host.double().square().sum(1).sqrt()
        worst = float(((norms[:, 0].double().cpu() - want).abs() / want).max())
        print(f"{dtype} {size}: worst {worst * 2 ** 24:.3f} half steps", flush=True)
        assert worst <= 2.0 ** -24 + 2.0 ** -40


def test_the_default_stream_by_its_handle_under_another():
    """stream=0 while another stream is current: the default stream's memory."""
    import lora_moe_amd as lm
    x, W_gu, W_down, _ = (t.cuda() for t in ffn_inputs(40, 136, 200, 3))
    want = lm.gated_ffn(x, W_gu, W_down)
    grads = lm.GradSet([torch.ones(100, device="cuda")])
    norm = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        y = lm.gated_ffn(x, W_gu, W_down, stream=0)
        lm.moe_lora_clip_grads(grads, math.inf, norm, stream=0)
    torch.cuda.synchronize()
    assert pool_of(y) == 0 and pool_of(grads._workspace(0)) == 0
    assert torch.equal(y, want) and float(norm) == 10.0

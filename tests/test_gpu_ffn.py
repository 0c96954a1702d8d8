"""The gated feed-forward block on the GPU: forward, kept pre-activations and
gradients against 64-bit forms, within bounds from the roundings."""
import pytest
import torch

from dense_common import HALF_BF16, act64, ffn64, ffn_backward_bounds, ffn_bounds, ffn_inputs, within

pytestmark = pytest.mark.gpu


def check_l2(l2, n, terms, what, roundings=2):
    """The relative L2 error of a result with one or two independent roundings
    to bf16 (of the sum, and of the summands): each is at most 2^-8 / sqrt(3) of
    the value in the mean square (uniform within half a step), 1.3 for the
    spread.  It is a mean: over few elements or few summands a single result
    may err by its worst case, 2^-8 (1 + sum |terms| / |sum|), which passes
    any such mean (at 8 elements of 8 terms 4.6e-3 against 4.1e-3), so it is
    asked of 4096 elements of 64 terms on; the bound per element holds
    everywhere."""
    if n >= 4096 and terms >= 64:
        assert l2 <= 1.3 * HALF_BF16 * (roundings / 3) ** 0.5, (what, l2)


def forward(lm, x, W_gu, W_down, act, keep=False, ws=None, stream=None):
    T, H = x.shape
    I = W_down.shape[1]
    shape = lm.make_ffn_shape(T, H, I, act)
    ws = lm.alloc_ffn_workspace(shape) if ws is None else ws
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    gu = torch.full((T, 2 * I), float("nan"), device="cuda") if keep else None
    lm.moe_lora_ffn_forward(shape, x, W_gu, W_down, ws, y, gu=gu, stream=stream)
    return shape, ws, y, gu


def gradients(lm, shape, ws, dy, x, gu, W_gu, W_down, want=("dx", "dW_gu", "dW_down"), stream=None):
    like = dict(dx=x, dW_gu=W_gu, dW_down=W_down)
    out = {n: torch.full_like(like[n], float("nan")) for n in want}
    lm.moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, ws, stream=stream, **out)
    return out


# one token to a few hundred, one off each tile edge, sizes that end inside
# 16-, 32-, 64-, 128- and 256-wide tiles and inside a K stage
SIZES = [(1, 8, 8), (1, 256, 512), (2, 264, 72), (7, 72, 1000), (16, 512, 256), (17, 104, 200), (31, 128, 64),
         (33, 1000, 328), (48, 640, 1288), (64, 256, 512), (65, 136, 520), (127, 392, 264), (129, 256, 136),
         (200, 776, 568), (255, 264, 1016), (257, 520, 392), (300, 1032, 776), (513, 256, 256)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_block(T, H, I, act):
    import lora_moe_amd as lm
    x, W_gu, W_down, dy = ffn_inputs(T, H, I, 100 * T + H)
    dx_, dg_, dd_, dyd = (t.cuda() for t in (x, W_gu, W_down, dy))
    shape, ws, y, gu = forward(lm, dx_, dg_, dd_, act, keep=True)
    (gu64, _, y64), (e_gu, _, e_y) = ffn_bounds(x.double(), W_gu.double(), W_down.double(), act)
    what = f"T={T} H={H} I={I} {act}"
    within(gu, gu64, e_gu, what + " gu")
    l2 = within(y, y64, e_y, what + " y")
    check_l2(l2, y.numel(), I, what)
    # the forward that keeps nothing may take other kernels (few tokens)
    y_inf = forward(lm, dx_, dg_, dd_, act)[2]
    within(y_inf, y64, e_y, what + " y, nothing kept")
    assert torch.equal(forward(lm, dx_, dg_, dd_, act)[2], y_inf)
    got = gradients(lm, shape, ws, dyd, dx_, gu, dg_, dd_)
    want = ffn_backward_bounds(dy.double(), x.double(), gu.double().cpu(), W_gu.double(), W_down.double(), act)
    for n, (v, e) in want.items():
        l2 = within(got[n], v, e, f"{what} {n}")
        # up to 16 tokens the summands carry their remainders, whatever their number
        if T <= 16:
            check_l2(l2, got[n].numel(), 64, f"{what} {n}", 1)
        else:
            check_l2(l2, got[n].numel(), 2 * I if n == "dx" else T, f"{what} {n}")
    again = gradients(lm, shape, ws, dyd, dx_, gu, dg_, dd_)
    for n in got:
        assert torch.equal(got[n], again[n]), n  # the same bits every time


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """<gradient, d> against the 64-bit central difference of <dy, y> along
    d: the difference's own error is of order step^2 (1e-8 here), the
    gradient's bound is summed over the elements."""
    import lora_moe_amd as lm
    T, H, I = 37, 72, 104
    x, W_gu, W_down, dy = ffn_inputs(T, H, I, 5)
    dev = [t.cuda() for t in (x, W_gu, W_down, dy)]
    shape, ws, _, gu = forward(lm, *dev[:3], act, keep=True)
    got = gradients(lm, shape, ws, dev[3], dev[0], gu, dev[1], dev[2])
    p64 = dict(dx=x.double(), dW_gu=W_gu.double(), dW_down=W_down.double())
    bounds = ffn_backward_bounds(dy.double(), *(p64["dx"], gu.double().cpu()), p64["dW_gu"], p64["dW_down"], act)
    gen = torch.Generator().manual_seed(9)
    for n in p64:
        d = torch.randn(p64[n].shape, generator=gen, dtype=torch.float64)
        d /= d.norm()
        def loss(t):
            q = dict(p64)
            q[n] = p64[n] + t * d
            return float((dy.double() * ffn64(q["dx"], q["dW_gu"], q["dW_down"], act)[2]).sum())
        step = 1e-4
        diff = (loss(step) - loss(-step)) / (2 * step)
        inner = float((got[n].double().cpu() * d).sum())
        tol = float((bounds[n][1] * d.abs()).sum()) + 1e-6
        print(f"{n}: {inner:.6e} against {diff:.6e}, tolerance {tol:.1e}", flush=True)
        assert abs(inner - diff) <= tol


@pytest.mark.parametrize("want", [("dx",), ("dW_gu",), ("dW_down",), ("dx", "dW_down")])
def test_wanted_gradients_only(want):
    """A frozen weight's gradient is not computed; the others keep their bits."""
    import lora_moe_amd as lm
    dev = [t.cuda() for t in ffn_inputs(70, 136, 200, 3)]
    x, W_gu, W_down, dy = dev
    shape, ws, _, gu = forward(lm, x, W_gu, W_down, "silu", keep=True)
    full = gradients(lm, shape, ws, dy, x, gu, W_gu, W_down)
    part = gradients(lm, shape, ws, dy, x, gu, W_gu, W_down, want)
    assert set(part) == set(want)
    for n in want:
        assert torch.equal(part[n], full[n])


def test_no_tokens():
    """T = 0: nothing to do forward, weight gradients of zero backward."""
    import lora_moe_amd as lm
    H, I = 72, 40
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    _, W_gu, W_down, _ = (t.cuda() for t in ffn_inputs(1, H, I, 1))
    shape, ws, y, gu = forward(lm, e, W_gu, W_down, "silu", keep=True)
    got = gradients(lm, shape, ws, e, e, gu, W_gu, W_down)
    assert not got["dW_gu"].any() and not got["dW_down"].any()


def test_no_tokens_dx_only():
    """T = 0 with an empty dx as the only gradient is nothing to do."""
    import lora_moe_amd as lm
    H, I = 72, 40
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    _, W_gu, W_down, _ = (t.cuda() for t in ffn_inputs(1, H, I, 1))
    shape = lm.make_ffn_shape(0, H, I)
    ws = lm.alloc_ffn_workspace(shape)
    gu = torch.empty((0, 2 * I), device="cuda")
    lm.moe_lora_ffn_backward(shape, e, e, gu, W_gu, W_down, ws, dx=torch.empty_like(e))


@pytest.mark.parametrize("T", [1, 6, 16, 20])
def test_infinities_stay_infinite(T):
    """Where h or a gradient leaves bf16's range the outputs are the formula's
    infinities, also where values go on as pairs (up to 16 tokens)."""
    import lora_moe_amd as lm
    H, I = 64, 64
    x = torch.full((T, H), 2.0 ** 62, dtype=torch.bfloat16, device="cuda")
    W_gu = torch.full((2 * I, H), 0.25, dtype=torch.bfloat16, device="cuda")
    W_down = torch.full((H, I), 0.5, dtype=torch.bfloat16, device="cuda")
    # g = u = 2^66: h = 2^132 is past every range
    shape, ws, y, gu = forward(lm, x, W_gu, W_down, "silu", keep=True)
    assert (gu == 2.0 ** 66).all() and (y == float("inf")).all()
    dy = torch.full((T, H), 2.0 ** 62, dtype=torch.bfloat16, device="cuda")
    got = gradients(lm, shape, ws, dy, x, gu, W_gu, W_down)
    for n, t in got.items():  # dh = 2^67, dg = dh u and du = dh g likewise
        assert (t == float("inf")).all(), n


def test_extreme_gates():
    """Pre-activations far out on both sides: the gate saturates, nothing
    overflows on the way (gelu's cube, exp)."""
    import lora_moe_amd as lm
    T, H, I = 16, 64, 64
    for act in ("silu", "gelu"):
        for scale in (1e3, 1e6):
            x, W_gu, W_down, dy = ffn_inputs(T, H, I, 21, scale)
            dev = [t.cuda() for t in (x, W_gu, W_down, dy)]
            shape, ws, y, gu = forward(lm, *dev[:3], act, keep=True)
            got = gradients(lm, shape, ws, dev[3], dev[0], gu, dev[1], dev[2])
            g64 = gu.double().cpu()
            a, da = act64(g64[:, :I], act)
            want = (a * g64[:, I:]) @ W_down.double().T
            # three roundings of h, y and the gate's own; of the sum's size
            tol = 3 * HALF_BF16 * ((a * g64[:, I:]).abs() @ W_down.double().abs().T)
            within(y, want, tol, f"{act} scale {scale:g}")
            for n in got:
                assert torch.isfinite(got[n]).all(), (act, scale, n)


def test_rows_are_their_own():
    """A token's output does not depend on the others: a row of NaN and a row
    of infinities stay in their rows."""
    import lora_moe_amd as lm
    for T in (5, 40, 150, 300):
        x, W_gu, W_down, _ = ffn_inputs(T, 136, 264, 4)
        dev = [t.cuda() for t in (x, W_gu, W_down)]
        y = forward(lm, *dev, "silu")[2]
        bad = dev[0].clone()
        bad[1] = float("nan")
        bad[T - 2] = float("inf")
        yb = forward(lm, bad, *dev[1:], "silu")[2]
        keep = torch.ones(T, dtype=torch.bool)
        keep[[1, T - 2]] = False
        assert torch.equal(yb[keep.cuda()], y[keep.cuda()])
        assert not torch.isfinite(yb[1]).any()


def test_memory_around_is_left_alone():
    """Outputs inside a larger buffer: the bytes before and behind stay, and
    NaN around the inputs never enters (sizes that end inside every tile)."""
    import lora_moe_amd as lm
    for T in (3, 61, 131):
        H, I, pad = 136, 72, 512
        src = [t.cuda() for t in ffn_inputs(T, H, I, 8)]
        def inside(t, fill):
            buf = torch.full((t.numel() + 2 * pad,), fill, dtype=t.dtype, device="cuda")
            v = buf[pad:pad + t.numel()].view(t.shape)
            return buf, v
        ins = []
        for t in src:
            buf, v = inside(t, float("nan"))
            v.copy_(t)
            ins.append(v)
        x, W_gu, W_down, dy = ins
        shape = lm.make_ffn_shape(T, H, I)
        nws = lm.moe_lora_ffn_workspace_bytes(shape)
        wsb = torch.full((nws + 1024,), 0xAB, dtype=torch.uint8, device="cuda")
        outs = {n: inside(t, 7.0) for n, t in (("y", x), ("dx", x), ("dW_gu", W_gu), ("dW_down", W_down))}
        gub, gu = inside(torch.empty((T, 2 * I), device="cuda"), 7.0)
        lm.moe_lora_ffn_forward(shape, x, W_gu, W_down, wsb[512:512 + nws], outs["y"][1], gu=gu)
        lm.moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, wsb[512:512 + nws],
                                 **{n: outs[n][1] for n in ("dx", "dW_gu", "dW_down")})
        ref = forward(lm, *src[:3], "silu", keep=True)
        n_inf = lm.moe_lora_ffn_workspace_bytes(shape, False)
        wsi = torch.full((n_inf + 1024,), 0xAB, dtype=torch.uint8, device="cuda")
        yib, yi = inside(src[0], 7.0)
        lm.moe_lora_ffn_forward(shape, x, W_gu, W_down, wsi[512:512 + n_inf], yi)
        assert torch.equal(yi, forward(lm, *src[:3], "silu")[2])
        assert (yib[:pad] == 7).all() and (yib[-pad:] == 7).all()
        assert (wsi[:512] == 0xAB).all() and (wsi[512 + n_inf:] == 0xAB).all()
        assert torch.equal(ref[2], outs["y"][1]) and torch.equal(ref[3], gu)
        grads = gradients(lm, ref[0], ref[1], src[3], src[0], ref[3], src[1], src[2])
        for n in grads:
            assert torch.equal(grads[n], outs[n][1]), n
        for n, (buf, _) in list(outs.items()) + [("gu", (gub, gu))]:
            assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all(), n
        assert (wsb[:512] == 0xAB).all() and (wsb[512 + nws:] == 0xAB).all()


@pytest.mark.parametrize("T", [3, 48, 200])
def test_graph_replays(T):
    """Forward and backward captured together; replays on changed inputs, with
    eager work of the same block between them, match eager runs bit for bit."""
    import lora_moe_amd as lm
    H, I = 264, 328
    x, W_gu, W_down, dy = (t.cuda() for t in ffn_inputs(T, H, I, 6))
    shape, ws, y, gu = forward(lm, x, W_gu, W_down, "gelu", keep=True)
    out = gradients(lm, shape, ws, dy, x, gu, W_gu, W_down)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        lm.moe_lora_ffn_forward(shape, x, W_gu, W_down, ws, y, gu=gu, stream=s)
        lm.moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, ws, stream=s, **out)
    for rep in range(3):
        x2, _, _, dy2 = (t.cuda() for t in ffn_inputs(T, H, I, 60 + rep))
        e_shape, e_ws, ey, egu = forward(lm, x2, W_gu, W_down, "gelu", keep=True)
        eg = gradients(lm, e_shape, e_ws, dy2, x2, egu, W_gu, W_down)
        x.copy_(x2)
        dy.copy_(dy2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(gu, egu), rep
        for n in out:
            assert torch.equal(out[n], eg[n]), (rep, n)


def test_two_streams():
    """Two blocks at once on two streams, each with its own workspace."""
    import lora_moe_amd as lm
    jobs = []
    for T, H, I, act in ((150, 264, 328, "silu"), (5, 512, 1000, "gelu")):
        x, W_gu, W_down, dy = (t.cuda() for t in ffn_inputs(T, H, I, T))
        shape, ws, y, gu = forward(lm, x, W_gu, W_down, act, keep=True)
        ref = gradients(lm, shape, ws, dy, x, gu, W_gu, W_down)
        jobs.append((shape, ws, x, W_gu, W_down, dy, y, gu, ref, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for shape, ws, x, W_gu, W_down, dy, y, gu, ref, s in jobs:
            s.wait_stream(torch.cuda.current_stream())
            y2, gu2 = torch.empty_like(y), torch.empty_like(gu)
            out = {n: torch.empty_like(t) for n, t in ref.items()}
            s.wait_stream(torch.cuda.current_stream())
            lm.moe_lora_ffn_forward(shape, x, W_gu, W_down, ws, y2, gu=gu2, stream=s)
            lm.moe_lora_ffn_backward(shape, dy, x, gu2, W_gu, W_down, ws, stream=s, **out)
            got.append((y2, gu2, out))
        torch.cuda.synchronize()
        for (y2, gu2, out), job in zip(got, jobs):
            assert torch.equal(y2, job[6]) and torch.equal(gu2, job[7])
            for n in out:
                assert torch.equal(out[n], job[8][n]), n


def test_one_call_form():
    import lora_moe_amd as lm
    x, W_gu, W_down, _ = (t.cuda() for t in ffn_inputs(20, 136, 72, 2))
    assert torch.equal(lm.gated_ffn(x, W_gu, W_down, act="gelu"), forward(lm, x, W_gu, W_down, "gelu")[2])


# sizes at which each product takes the large tiles, ending inside them, and
# few tokens with more weight-gradient tiles than one grid takes
@pytest.mark.parametrize("T,H,I,act", [(2050, 2072, 4104, "silu"), (4200, 2056, 2008, "gelu"),
                                       (13, 2056, 5512, "silu"), (40, 2056, 5512, "gelu")])
def test_large_block(T, H, I, act):
    """The same bounds with the 64-bit products formed on the GPU."""
    import lora_moe_amd as lm
    x, W_gu, W_down, dy = (t.cuda() for t in ffn_inputs(T, H, I, 17))
    shape, ws, y, gu = forward(lm, x, W_gu, W_down, act, keep=True)
    got = gradients(lm, shape, ws, dy, x, gu, W_gu, W_down)
    d = [t.double() for t in (x, W_gu, W_down, dy)]
    (gu64, _, y64), (e_gu, _, e_y) = ffn_bounds(*d[:3], act)
    want = ffn_backward_bounds(d[3], d[0], gu.double(), d[1], d[2], act)
    want["gu"], want["y"] = (gu64, e_gu), (y64, e_y)
    got.update(gu=gu, y=y)
    for n, (v, e) in want.items():
        l2 = within(got[n], v.cpu(), e.cpu(), f"T={T} H={H} I={I} {n}")
        if n != "gu":
            check_l2(l2, v.numel(), T, n)

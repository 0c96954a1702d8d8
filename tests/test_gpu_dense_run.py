"""The dense operators together, as a program uses them: training steps of a
gated block (forward, backward, clipping, an update of the weights), then the
trained weights in 4 bits in a decode loop.  Each stage is held against its
64-bit form on the values that the stage before it left."""
import math

import pytest
import torch

from dense_common import (HALF_BF16, HALF_F32, LIP, act64, ffn_backward_bounds, ffn_bounds, ffn_inputs, w4_bounds,
                          w4_values, within)

pytestmark = pytest.mark.gpu

T, H, I, GROUP = 70, 136, 200, 64
MAX_NORM, RATE = 0.05, 2.0


class Block:
    """A block's weights, gradients and buffers; step() is one training step
    towards a target with the loss |y - target|^2 / 2."""

    def __init__(self, lm, tokens, seed):
        self.lm = lm
        x, W_gu, W_down, target = (t.cuda() for t in ffn_inputs(tokens, H, I, seed))
        self.x, self.target = x, target
        self.W = [W_gu, W_down]
        self.master = [w.float() for w in self.W]
        self.shape = lm.make_ffn_shape(tokens, H, I)
        self.ws = lm.alloc_ffn_workspace(self.shape)
        self.y, self.dy, self.dx = (torch.empty_like(x) for _ in range(3))
        self.gu = torch.empty((tokens, 2 * I), device="cuda")
        self.dW = [torch.empty_like(w) for w in self.W]
        self.clipped = [torch.empty_like(w) for w in self.W]
        self.grads = lm.GradSet(self.dW, out=self.clipped)
        self.norm = torch.empty(1, device="cuda")

    def step(self):
        lm = self.lm
        lm.moe_lora_ffn_forward(self.shape, self.x, *self.W, self.ws, self.y, gu=self.gu)
        torch.sub(self.y, self.target, out=self.dy)
        lm.moe_lora_ffn_backward(self.shape, self.dy, self.x, self.gu, *self.W, self.ws, dx=self.dx,
                                 dW_gu=self.dW[0], dW_down=self.dW[1])
        lm.moe_lora_clip_grads(self.grads, MAX_NORM, self.norm)
        for w, m, g in zip(self.W, self.master, self.clipped):
            m.sub_(g, alpha=RATE)
            w.copy_(m)

    def check(self, W, what):
        """The last step's values, from the weights W (64 bits) before it."""
        d = [t.double().cpu() for t in (self.x, self.dy, self.gu)]
        (gu, _, y), (e_gu, _, e_y) = ffn_bounds(d[0], *W, "silu")
        within(self.gu, gu, e_gu, f"{what} gu")
        within(self.y, y, e_y, f"{what} y")
        want = ffn_backward_bounds(d[1], d[0], d[2], *W, "silu")
        for n, t in (("dx", self.dx), ("dW_gu", self.dW[0]), ("dW_down", self.dW[1])):
            within(t, *want[n], f"{what} {n}")
        g = [t.double().cpu() for t in self.dW]
        norm = math.sqrt(sum(float((t * t).sum()) for t in g))
        # the norm's fp32 rounding, and that of each 16-byte piece's sum (7 additions, 8 squares)
        assert abs(float(self.norm) - norm) <= 10 * HALF_F32 * norm, what
        c = min(1.0, MAX_NORM / (norm + 1e-6))
        for t, o in zip(g, self.clipped):
            # c and the product in fp32, then bf16
            within(o, t * c, (HALF_BF16 + 16 * HALF_F32) * (t * c).abs(), f"{what} clipped")


def quantise(w):
    """Round to nearest in 4 bits per row and group of GROUP, with zero points."""
    n, k = w.shape
    G = (k + GROUP - 1) // GROUP
    p = torch.zeros((n, G * GROUP))
    p[:, :k] = w.float().cpu()
    p = p.view(n, G, GROUP)
    lo, hi = p.amin(2).clamp(max=0), p.amax(2).clamp(min=0)
    s = ((hi - lo) / 15).clamp(min=1e-8).bfloat16()
    z = (-lo / s.float()).round().clamp(0, 15)
    q = (p / s.float()[..., None] + z[..., None]).round().clamp(0, 15).to(torch.uint8).view(n, G * GROUP)[:, :k]
    return (q[:, 0::2] | q[:, 1::2] << 4).contiguous(), s, z.to(torch.uint8)


def w4_block_bounds(x, values):
    """The 4-bit block in 64 bits with the bound on its roundings."""
    g, e_g, _ = w4_bounds(x, *values["gate"])
    u, e_u, _ = w4_bounds(x, *values["up"])
    a, _ = act64(g, "silu")
    h = a * u
    e_a = LIP * e_g + 64 * HALF_F32 * (a.abs() + g.abs())
    e_h = e_a * u.abs() + (a.abs() + e_a) * e_u
    e_h = e_h + HALF_BF16 * (h.abs() + e_h)
    want, e, _ = w4_bounds(h, *values["down"])
    e = e * 1.01 + e_h @ values["down"][0].abs().T + (I + 8) * HALF_F32 * (e_h @ values["down"][1].T)
    return want, e + HALF_BF16 * (want.abs() + e)


@pytest.mark.parametrize("tokens", [T, 9])
def test_train_then_decode_in_4_bits(tokens):
    import lora_moe_amd as lm
    b = Block(lm, tokens, 5)
    for i in range(3):
        W = [w.double().cpu() for w in b.W]
        b.step()
        b.check(W, f"step {i}")
    parts = {"gate": quantise(b.W[0][:I]), "up": quantise(b.W[0][I:]), "down": quantise(b.W[1])}
    w = {n: lm.moe_lora_w4_pack(*(t.cuda() for t in p), group=GROUP) for n, p in parts.items()}
    values = {n: w4_values(*p, GROUP) for n, p in parts.items()}
    for n, orig in (("gate", b.W[0][:I]), ("up", b.W[0][I:]), ("down", b.W[1])):
        # half a step of 4 bits, and at the ends that of the zero point and the scale's own over 15 steps
        s = parts[n][1].double().repeat_interleave(GROUP, 1)[:, :orig.shape[1]]
        assert ((values[n][0] - orig.double().cpu()).abs() <= (0.5 + 0.5 + 16 * HALF_BF16) * s).all(), n
    for M in (1, 7):
        x, ws = b.x[:M].contiguous(), lm.alloc_w4_ffn_workspace(M, I)
        for i in range(3):
            y = torch.empty_like(x)
            lm.moe_lora_w4_ffn_forward(x, w["gate"], w["up"], w["down"], ws, y)
            want, bound = w4_block_bounds(x.double().cpu(), values)
            within(y, want, bound, f"M={M} decode {i}")
            x = (x + y).contiguous()  # a residual stream


def test_captured_step_and_decode():
    """A training step and a 4-bit decode step captured in one graph; every
    replay, with eager work of the same kind between, gives the bits of an
    eager run."""
    import lora_moe_amd as lm
    a, e = Block(lm, T, 8), Block(lm, T, 8)
    q = [lm.moe_lora_w4_pack(*(t.cuda() for t in quantise(m)), group=GROUP)
         for m in (a.W[0][:I], a.W[0][I:], a.W[1])]
    ws = [lm.alloc_w4_ffn_workspace(4, I) for _ in range(2)]
    xs = [a.x[:4].clone() for _ in range(2)]
    ys = [torch.empty_like(xs[0]) for _ in range(2)]

    def both(b, i):
        b.step()
        lm.moe_lora_w4_ffn_forward(xs[i], *q, ws[i], ys[i])
        xs[i].add_(ys[i])

    state = [t.clone() for t in a.W + a.master]
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        both(a, 0)
    for t, k in zip(a.W + a.master, state):  # (capturing ran nothing)
        assert torch.equal(t, k)
    for rep in range(4):
        both(e, 1)
        g.replay()
        torch.cuda.synchronize()
        for n in ("y", "dx", "gu", "norm"):
            assert torch.equal(getattr(a, n), getattr(e, n)), (rep, n)
        for n in ("W", "master", "dW", "clipped"):
            for t, k in zip(getattr(a, n), getattr(e, n)):
                assert torch.equal(t, k), (rep, n)
        assert torch.equal(ys[0], ys[1]) and torch.equal(xs[0], xs[1]), rep


def test_default_stream_by_its_handle():
    """stream=0, the default stream's handle, and a Stream object give the
    same results as no stream."""
    import lora_moe_amd as lm
    x, W_gu, W_down, _ = (t.cuda() for t in ffn_inputs(5, H, I, 2))
    ref = lm.gated_ffn(x, W_gu, W_down)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [lm.gated_ffn(x, W_gu, W_down, stream=st) for st in (0, s, s.cuda_stream)]
    torch.cuda.synchronize()
    for t in got:
        assert torch.equal(t, ref)

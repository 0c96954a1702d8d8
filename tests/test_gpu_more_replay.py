"""The operators around the routed experts captured into graphs: a fine-tuning
step whose run lengths the program holds, and a decode loop of two projections
with the routed layer between them.  Every replay is held against the eager
result, bit for bit, with eager work between the replays."""
import pytest
import torch

import lora_moe_amd as lm
from dense_common import within
from proj_common import forward64
from test_gpu_more_run import E, K, L, R, T, Layer, bf16

pytestmark = pytest.mark.gpu


class Step(Layer):
    """Runs of fixed lengths, buffers and workspaces made once."""

    def __init__(self, seed):
        super().__init__(seed)
        self.forward()
        self.fixed = self.off.tolist()
        runs = [b - a for a, b in zip(self.fixed, self.fixed[1:])]
        self.block = [(s, lm.alloc_ffn_workspace(s)) for s in (lm.make_ffn_shape(n, self.W.shape[0], 64) for n in runs)]

    def experts(self, backward):
        if not hasattr(self, "block"):
            return super().experts(backward)
        for e, (s, ws) in enumerate(self.block):
            a, b = self.fixed[e], self.fixed[e + 1]
            if not backward:
                lm.moe_lora_ffn_forward(s, self.rows[a:b], self.W_gu[e], self.W_down[e], ws, self.d[a:b],
                                        gu=self.gu[a:b])
            else:
                lm.moe_lora_ffn_backward(s, self.dd[a:b], self.rows[a:b], self.gu[a:b], self.W_gu[e], self.W_down[e],
                                         ws, dx=self.drows[a:b], dW_gu=self.dW[e][0], dW_down=self.dW[e][1])
        return self.fixed

    def step(self):
        self.forward()
        self.backward()
        lm.moe_lora_clip_grads(self.grads, 0.5, self.norm)

    def outputs(self):
        return [self.q, self.z, self.topk, self.weights, self.off, self.row, self.rows, self.d, self.y, self.dd, self.dw,
                self.drows, self.dq, self.dlogits, self.dx, self.dA, self.dB, self.norm] + [t for p in self.dW for t in p]


def test_a_captured_step_repeats_the_eager_one():
    layer, other = Step(7), Step(8)
    g = torch.Generator().manual_seed(3)
    # (powers of two, which leave the experts' choice as it is)
    inputs = [(layer.x * f, bf16(g, *layer.target.shape)) for f in (2.0, 0.5, 1.0)]
    want = []
    for x, target in inputs:
        layer.x.copy_(x)
        layer.target.copy_(target)
        layer.step()
        assert layer.off.tolist() == layer.fixed
        want.append([t.clone() for t in layer.outputs()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    for n in (0, 1, 2, 0, 2):
        layer.x.copy_(inputs[n][0])
        layer.target.copy_(inputs[n][1])
        for t in layer.outputs():
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for i, (got, w) in enumerate(zip(layer.outputs(), want[n])):
            assert torch.equal(got, w), (n, i)
        other.step()  # eager work on buffers of its own
        torch.cuda.synchronize()


def test_a_decode_loop():
    """Four steps of x + P2(layer(P1(x))) for a batch of requests with adapters
    of their own, eager and replayed."""
    B, H, N, I = 6, 72, 128, 64
    g = torch.Generator().manual_seed(5)
    ids = torch.tensor([0, 2, -1, 1, 2, 0], dtype=torch.int32, device="cuda")
    scales = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    P = [(bf16(g, n, k, std=k ** -0.5), bf16(g, L, R, k, std=k ** -0.5), bf16(g, L, n, R, std=R ** -0.5))
         for k, n in ((H, N), (N, H))]
    shapes = [lm.make_proj_shape(B, H, N, L, R, 0.5), lm.make_proj_shape(B, N, H, L, R, 0.5)]
    ws = [lm.alloc_proj_workspace(s, backward=False) for s in shapes]
    s = lm.make_shape(B, N, I, E, K, L, 8)
    layer = [bf16(g, *n, std=n[-1] ** -0.5) for n in
             ((E, 2 * I, N), (E, N, I), (L, E, 8, N), (L, E, 2 * I, 8), (L, E, 8, I), (L, E, N, 8))]
    layer_ws, router = lm.alloc_workspace(s), torch.randn((E, N), generator=g).cuda() * N ** -0.5
    e = lambda n, t=torch.bfloat16: torch.empty((B, n), dtype=t, device="cuda")  # noqa: E731
    x, q, o, p = e(H), e(N), e(N), e(H)
    topk, weights = e(K, torch.int32), e(K, torch.float32)
    used = [e(H), e(N), e(N), e(H)]

    def step():
        used[0].copy_(x)
        lm.moe_lora_proj_forward(shapes[0], x, ids, *P[0], ws[0], q, scales=scales)
        lm.moe_lora_route(s, q.float() @ router.T, topk, weights)
        lm.moe_lora_align(s, topk, ids, layer_ws)
        lm.moe_lora_forward(s, q, topk, weights, ids, *layer, layer_ws, o)
        lm.moe_lora_proj_forward(shapes[1], o, ids, *P[1], ws[1], p, scales=scales)
        x.add_(p)

    first = bf16(g, B, H)
    want = []
    x.copy_(first)
    for _ in range(4):
        step()
        want.append([t.clone() for t in (used[0], q, o, p, x)])
        c = [[t.double().cpu() for t in (v, *w)] for v, w in ((used[0], P[0]), (o, P[1]))]
        within(q, *forward64(*c[0], ids.cpu(), scales.cpu(), 0.5)[1], "P1")
        within(p, *forward64(*c[1], ids.cpu(), scales.cpu(), 0.5)[1], "P2")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        x.copy_(first)
        for n in range(4):
            for t in (q, o, p):
                t.fill_(1)
            graph.replay()
            torch.cuda.synchronize()
            for got, w in zip((used[0], q, o, p, x), want[n]):
                assert torch.equal(got, w), n
            lm.lora_projection(first, ids, *P[0], 0.5, scales=scales)

"""The operators around the routed experts together, as a fine-tuning step uses
them: a shared projection with several adapters, the router, the tokens sorted
to their experts, each expert's gated block on its run, back with the router's
weights, and all of it backwards into the adapters' gradients, which are clipped
and applied.  Each stage is held against its 64-bit form on the values that the
stage before it left; then a decode batch runs on the trained adapters."""
import math

import pytest
import torch

import lora_moe_amd as lm
from dense_common import HALF_BF16, HALF_F32, ffn_backward_bounds, ffn_bounds, within
from proj_common import backward64, forward64, inputs

pytestmark = pytest.mark.gpu

T, H, N, I, E, K, L, R = 90, 72, 136, 64, 5, 2, 3, 16


def bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).bfloat16().cuda()


class Layer:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        x, W, A, B, _, ids, scales = inputs(T, H, N, L, R, seed, "runs")
        self.x, self.W, self.A, self.B, self.ids, self.scales = (t.cuda() for t in (x, W, A, B, ids, scales))
        self.master = [t.float() for t in (self.A, self.B)]
        self.router = torch.randn((E, N), generator=g).cuda() * N ** -0.5
        self.W_gu = [bf16(g, 2 * I, N, std=N ** -0.5) for _ in range(E)]
        self.W_down = [bf16(g, N, I, std=I ** -0.5) for _ in range(E)]
        self.target = bf16(g, T, N)
        self.proj, self.sort = lm.make_proj_shape(T, H, N, L, R, 0.5), lm.make_sort_shape(T, N, E, K)
        self.route = lm.make_shape(T, N, I, E, K, 1, 8)
        self.ws, self.sort_ws = lm.alloc_proj_workspace(self.proj), lm.alloc_sort_workspace(self.sort)
        e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        f32, i32 = torch.float32, torch.int32
        self.q, self.z = e(T, N), e(T, R, t=f32)
        self.topk, self.weights = e(T, K, t=i32), e(T, K, t=f32)
        self.rows, self.d, self.dd, self.drows = (e(T * K, N) for _ in range(4))
        self.off, self.row = e(E + 1, t=i32), e(T, K, t=i32)
        self.y, self.dy, self.dq, self.dx = e(T, N), e(T, N), e(T, N), e(T, H)
        self.dw, self.dlogits = e(T, K, t=f32), e(T, E, t=f32)
        self.dA, self.dB = torch.empty_like(self.A), torch.empty_like(self.B)
        self.grads, self.norm = lm.GradSet([self.dA, self.dB]), e(1, t=f32)
        self.gu = e(T * K, 2 * I, t=f32)
        self.dW = [(torch.empty_like(a), torch.empty_like(b)) for a, b in zip(self.W_gu, self.W_down)]

    def experts(self, backward):
        runs = self.off.tolist()
        assert runs[-1] == T * K
        for e in range(E):
            a, b = runs[e], runs[e + 1]
            s = lm.make_ffn_shape(b - a, N, I)
            ws = lm.alloc_ffn_workspace(s)
            if not backward:
                lm.moe_lora_ffn_forward(s, self.rows[a:b], self.W_gu[e], self.W_down[e], ws, self.d[a:b],
                                        gu=self.gu[a:b])
            else:
                lm.moe_lora_ffn_backward(s, self.dd[a:b], self.rows[a:b], self.gu[a:b], self.W_gu[e], self.W_down[e],
                                         ws, dx=self.drows[a:b], dW_gu=self.dW[e][0], dW_down=self.dW[e][1])
        return runs

    def forward(self):
        lm.moe_lora_proj_forward(self.proj, self.x, self.ids, self.W, self.A, self.B, self.ws, self.q, z=self.z,
                                 scales=self.scales)
        self.logits = self.q.float() @ self.router.T
        lm.moe_lora_route(self.route, self.logits, self.topk, self.weights)
        lm.moe_lora_sort(self.sort, self.topk, self.q, self.sort_ws, self.rows, self.off, self.row)
        self.runs = self.experts(False)
        lm.moe_lora_unsort(self.sort, self.d, self.row, self.y, weights=self.weights)

    def backward(self):
        torch.sub(self.y, self.target, out=self.dy)
        lm.moe_lora_unsort_backward(self.sort, self.dy, self.d, self.row, self.dd, weights=self.weights,
                                    dweights=self.dw)
        self.experts(True)
        lm.moe_lora_sort_backward(self.sort, self.drows, self.row, self.dq)
        lm.moe_lora_route_backward(self.route, self.topk, self.weights, self.dw, self.dlogits)
        self.into = (self.dq.float() + self.dlogits @ self.router).bfloat16()
        lm.moe_lora_proj_backward(self.proj, self.into, self.x, self.ids, self.z, self.W, self.A, self.B, self.ws,
                                  dx=self.dx, dA=self.dA, dB=self.dB, scales=self.scales)

    def update(self, rate):
        lm.moe_lora_clip_grads(self.grads, 0.5, self.norm)
        for p, m, g in zip((self.A, self.B), self.master, (self.dA, self.dB)):
            m.sub_(g, alpha=rate)
            p.copy_(m)

    def check(self):
        c = lambda *ts: [t.double().cpu() for t in ts]  # noqa: E731
        ids, scales = self.ids.cpu(), self.scales.cpu()
        x, W, A, B, q, z = c(self.x, self.W, self.A, self.B, self.q, self.z)
        (z64, e_z), (q64, e_q) = forward64(x, W, A, B, ids, scales, 0.5)
        within(self.z, z64, e_z, "z")
        within(self.q, q64, e_q, "q")
        # the sort: by expert, tokens in order, their rows bit for bit
        topk, row = self.topk.cpu().long(), self.row.cpu().long()
        flat = topk.reshape(-1)
        order = torch.argsort(flat, stable=True)
        assert torch.equal(row.reshape(-1)[order], torch.arange(T * K))
        assert self.runs == [int((flat < e).sum()) for e in range(E + 1)]
        assert torch.equal(self.rows.cpu(), self.q.cpu()[order // K])
        rows, d, w, dy, dd, drows = c(self.rows, self.d, self.weights, self.dy, self.dd, self.drows)
        for e in range(E):
            a, b = self.runs[e], self.runs[e + 1]
            if a == b:
                continue
            (gu, _, y), (e_gu, _, e_y) = ffn_bounds(rows[a:b], *c(self.W_gu[e], self.W_down[e]), "silu")
            within(self.gu[a:b], gu, e_gu, f"gu {e}")
            within(self.d[a:b], y, e_y, f"d {e}")
            want = ffn_backward_bounds(dd[a:b], rows[a:b], *c(self.gu[a:b], self.W_gu[e], self.W_down[e]), "silu")
            within(self.drows[a:b], *want["dx"], f"drows {e}")
            within(self.dW[e][0], *want["dW_gu"], f"dW_gu {e}")
            within(self.dW[e][1], *want["dW_down"], f"dW_down {e}")

        def near(got, terms, dim, half, what):
            v, size = terms.sum(dim), terms.abs().sum(dim)
            e = (terms.shape[dim] + 1) * HALF_F32 * size
            within(got, v, e + half * (v.abs() + e), what)

        near(self.y, d[row] * w[:, :, None], 1, HALF_BF16, "y")
        want = torch.zeros_like(dd)
        want[row.reshape(-1)] = (dy[:, None, :] * w[:, :, None]).reshape(T * K, N)
        within(self.dd, want, (HALF_BF16 + 2 * HALF_F32) * want.abs(), "dd")
        near(self.dw, d[row] * dy[:, None, :], 2, HALF_F32, "dweights")
        near(self.dq, drows[row], 1, HALF_BF16, "dq")
        dw = self.dw.double().cpu()
        s = (w * dw).sum(1, keepdim=True)
        e = w * ((K + 1) * (w * dw).abs().sum(1, keepdim=True) + 3 * (dw.abs() + s.abs())) * HALF_F32
        z0 = torch.zeros((T, E), dtype=torch.float64)
        within(self.dlogits, z0.scatter(1, topk, w * (dw - s)), z0.scatter(1, topk, 1.01 * e), "dlogits")
        grads = backward64(c(self.into)[0], x, z, W, A, B, ids, scales, 0.5)
        for n, t in (("dx", self.dx), ("dA", self.dA), ("dB", self.dB)):
            within(t, *grads[n], n)


def test_fine_tuning_steps():
    layer = Layer(7)
    for _ in range(2):
        layer.forward()
        layer.backward()
        torch.cuda.synchronize()
        layer.check()
        dA, dB = (t.double().cpu() for t in (layer.dA, layer.dB))
        old = [m.clone() for m in layer.master]
        layer.update(0.5)
        norm = math.sqrt(float((dA ** 2).sum() + (dB ** 2).sum()))
        assert abs(float(layer.norm) - norm) <= 4 * HALF_F32 * norm
        assert any(not torch.equal(m, o) for m, o in zip(layer.master, old))
    # a decode batch on the trained adapters: a token of each run and one without
    at = torch.tensor([0, 20, 45, 70, 89], device="cuda")
    x, ids = layer.x[at].contiguous(), layer.ids[at].contiguous()
    y = lm.lora_projection(x, ids, layer.W, layer.A, layer.B, 0.5, scales=layer.scales)
    c = [t.double().cpu() for t in (x, layer.W, layer.A, layer.B)]
    within(y, *forward64(*c, ids.cpu(), layer.scales.cpu(), 0.5)[1], "decode")

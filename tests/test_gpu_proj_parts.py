"""s_l z and u keep all bits of their fp32 sums on the way into the products
that follow them: whole numbers of 18 bits that differ in their last two, in
pairs whose large parts cancel, so that every result is exact."""
import pytest
import torch

import lora_moe_amd as lm

pytestmark = pytest.mark.gpu

LARGE = 2 ** 17 + 2 ** 8  # a bf16 and another; with an odd number behind them it takes three

# T, K (summed over), N, L, r: decode batches, and sorted ones that take each tile, whole and with K split
CASES = [(40, 72, 136, 3, 24), (300, 72, 520, 3, 8), (514, 136, 136, 3, 16), (520, 136, 72, 4, 128), (514, 8, 8, 2, 8),
         (2075, 752, 8, 3, 128), (2069, 8, 904, 5, 128), (1430, 3688, 8, 3, 128), (2235, 288, 3824, 4, 128),
         (1100, 264, 264, 1, 32), (5000, 136, 264, 2, 64)]


def whole(g, shape, p, most=1):
    return ((torch.rand(shape, generator=g) < p) * torch.randint(-most, most + 1, shape, generator=g)).double()


def alternating(g, ids, L, width, p):
    """Rows of which each second one of an adapter's tokens is the negative of
    the one before it (zeros where that has no partner)."""
    v = whole(g, (len(ids), width), p)
    for l in range(L):
        at = torch.nonzero(ids == l).flatten()
        n = len(at) // 2 * 2
        v[at[1:n:2]] = -v[at[0:n:2]]
        v[at[n:]] = 0
    return v


def down(g, T, L, width, r):
    """v [T, width] and w [L, r, width] with w v = LARGE and an odd number from 1
    to 5 for all pairs of token and rank."""
    v = whole(g, (T, width), 0.02)
    v[:, :4] = torch.tensor([2.0 ** 17, 2.0 ** 8, 1.0, 0.0])
    v[:, 3] = 2.0 * torch.randint(0, 2, (T,), generator=g)
    w = torch.zeros((L, r, width), dtype=torch.float64)
    w[:, :, :2] = 1
    w[:, :, 2] = 1.0 + 2 * torch.randint(0, 2, (L, r), generator=g)
    w[:, :, 3] = torch.randint(0, 2, (L, r), generator=g)
    return v, w


def back(g, L, out, r):
    """[L, out, r] whose neighbouring ranks are each other's negatives."""
    w = torch.zeros((L, out, r), dtype=torch.float64)
    w[:, :, 0::2] = whole(g, (L, out, r // 2), 0.2)
    w[:, :, 1::2] = -w[:, :, 0::2]
    return w


def shared(g, rows, columns):
    """[rows, columns] that the first two columns' large values do not meet."""
    W = whole(g, (rows, columns), 0.02)
    W[:, :4] = 0
    return W


def own(v, w, ids):
    y = torch.zeros((v.shape[0], w.shape[1]), dtype=torch.float64)
    for l in range(w.shape[0]):
        y[ids == l] = v[ids == l] @ w[l].T
    return y


def cuda(t, dtype=torch.bfloat16):
    assert torch.equal(t.to(dtype).double(), t)
    return t.to(dtype).cuda()


def same(got, want, what):
    assert float(want.abs().max()) <= 256 and bool(want.any()), what
    assert torch.equal(got.cpu().double(), want), what


@pytest.mark.parametrize("T,K,N,L,r", CASES)
def test_forward_keeps_all_bits_of_z(T, K, N, L, r):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, L, (T,), generator=g)
    x, A = down(g, T, L, K, r)
    W, B = shared(g, N, K), back(g, L, N, r)
    scales = torch.tensor([1.0, 2.0, -1.0, 1.0, 2.0])[:L]
    shape = lm.make_proj_shape(T, K, N, L, r)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((T, r), device="cuda")
    lm.moe_lora_proj_forward(shape, cuda(x), ids.int().cuda(), cuda(W), cuda(A), cuda(B), lm.alloc_proj_workspace(shape), y,
                             z=z, scales=scales.cuda())
    z64 = own(x, A, ids)
    assert torch.equal(z.cpu().double(), z64)
    s = torch.where(ids >= 0, scales[ids.clamp(min=0)], 0.0).double()[:, None]
    same(y, x @ W.T + own(s * z64, B, ids), "y")


@pytest.mark.parametrize("T,N,K,L,r", CASES)
def test_backward_keeps_all_bits_of_u_and_z(T, N, K, L, r):
    g = torch.Generator().manual_seed(T + 1)
    ids = torch.randint(-1, L, (T,), generator=g)
    dy, B = down(g, T, L, N, r)
    dy[:, 4:] = alternating(g, ids, L, N - 4, 0.05)
    x = alternating(g, ids, L, K, 0.05)
    W, A = shared(g, K, N).T.contiguous(), back(g, L, K, r).transpose(1, 2).contiguous()
    z = LARGE + 1.0 + 2 * torch.randint(0, 2, (T, r), generator=g).double()
    scales = torch.tensor([1.0, 2.0, -1.0, 1.0, 2.0])[:L]
    shape = lm.make_proj_shape(T, K, N, L, r)
    B = B.transpose(1, 2).contiguous()
    d = [cuda(t) for t in (dy, x, W, A, B)]
    dx, dA, dB = (torch.empty_like(d[i]) for i in (1, 3, 4))
    lm.moe_lora_proj_backward(shape, d[0], d[1], ids.int().cuda(), cuda(z, torch.float32), d[2], d[3], d[4],
                              lm.alloc_proj_workspace(shape), dx=dx, dA=dA, dB=dB, scales=scales.cuda())
    s = torch.where(ids >= 0, scales[ids.clamp(min=0)], 0.0).double()[:, None]
    u = own(s * dy, B.transpose(1, 2), ids)
    same(dx, dy @ W + own(u, A.transpose(1, 2), ids), "dx")
    for l in range(L):
        at = ids == l
        same(dA[l], u[at].T @ x[at], f"dA {l}")
        # (the large values of dy are not for here)
        same(dB[l, 4:], dy[at][:, 4:].T @ (s * z)[at], f"dB {l}")

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


@pytest.mark.parametrize("T,L", [(90, 6), (1500, 2)])
@pytest.mark.parametrize("r", [8, 24, 64, 128])
def test_gradients_of_rows_that_are_not_finite(T, L, r):
    """An infinity of x or dy is in the gradients what the formula makes of it,
    whether the values that it meets take one bf16 or three."""
    K, N, inf = 72, 136, float("inf")
    g = torch.Generator().manual_seed(r)
    r16 = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731
    x, dy, W, A, B = r16(T, K), r16(T, N), r16(N, K), r16(L, r, K), r16(L, N, r)
    z = torch.randn((T, r), generator=g)
    z[:, ::2] = (4 * z[:, ::2]).round() + 0.5  # (a bf16 each, and no 0)
    ids = (torch.arange(T) % L).int()
    shape = lm.make_proj_shape(T, K, N, L, r)
    ws = lm.alloc_proj_workspace(shape)

    def run(x, dy, **want):
        out = {n: torch.empty_like(t, device="cuda") for n, t in want.items()}
        lm.moe_lora_proj_backward(shape, dy.cuda(), x.cuda(), ids.cuda(), z.cuda(), W.cuda(), A.cuda(), B.cuda(), ws, **out)
        return [t.cpu() for t in out.values()]

    dA, dB = run(x, dy, dA=A, dB=B)
    u = own(dy.double(), B.double().transpose(1, 2), ids)
    sure = u.abs() > 1e-2  # (its sum in fp32 has this one's sign)
    x2, dy2 = x.clone(), dy.clone()
    a, b, c = L, 3 * L + 1, 4 * L + 1  # tokens of adapters 0 and 1
    x2[a, 5], x2[b, 7], x2[c, 7], x2[b, 11] = inf, -inf, -inf, float("nan")
    dA2, = run(x2, dy, dA=A)
    assert torch.equal(dA2[0][sure[a], 5], u[a][sure[a]].sign().float().mul(inf).bfloat16())
    two = sure[b] & sure[c]
    for j in torch.nonzero(two).flatten().tolist():
        want = float(-inf * u[b, j].sign() - inf * u[c, j].sign())
        assert torch.equal(dA2[1][j, 7].float(), torch.tensor(want)) or (want != want and bool(dA2[1][j, 7].isnan()))
    assert bool(dA2[1][:, 11].isnan().all())
    dA2[0][:, 5], dA2[1][:, 7], dA2[1][:, 11] = dA[0][:, 5], dA[1][:, 7], dA[1][:, 11]
    assert torch.equal(dA2, dA)
    dy2[a, 9], dy2[b, 100] = -inf, inf
    dB2, = run(x, dy2, dB=B)
    assert torch.equal(dB2[0][9], z[a].sign().mul(-inf).bfloat16())
    assert torch.equal(dB2[1][100], z[b].sign().mul(inf).bfloat16())
    dB2[0][9], dB2[1][100] = dB[0][9], dB[1][100]
    assert torch.equal(dB2, dB)
    z[a] = inf  # and infinities of both
    dB3, = run(x, dy2, dB=B)
    assert torch.equal(dB3[0][9], torch.full((r,), -inf, dtype=torch.bfloat16))

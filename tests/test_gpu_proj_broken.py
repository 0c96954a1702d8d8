"""Infinities and NaN of the adapters' weights in every form of the
projection's product: on whole numbers each output is exactly what the formula
gives, an infinity times an infinity among them."""
import pytest
import torch

import lora_moe_amd as lm
from proj_forms import SIZES

pytestmark = pytest.mark.gpu

CASES = [(9, 72, 136, 3, 16), (60, 136, 264, 5, 24), (300, 72, 520, 3, 8), *SIZES]  # (decode batches first)


def whole(g, shape, p, most=1):
    return ((torch.rand(shape, generator=g) < p) * torch.randint(-most, most + 1, shape, generator=g)).double()


def own(v, w, ids):
    """w[l_t] v_t with every term in it, the adapters one after the other."""
    y = torch.zeros((v.shape[0], w.shape[1]), dtype=torch.float64)
    for l in range(w.shape[0]):
        at = torch.nonzero(ids == l).flatten()
        if len(at):
            y[at] = v[at] @ w[l].T
    return y


def same(got, want, what):
    got, fine = got.cpu().double(), want.isfinite()
    assert float(want[fine].abs().max()) <= 256, what
    wrong = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bool(wrong.any()), (what, torch.nonzero(wrong)[:5].tolist(), got[wrong][:5], want[wrong][:5])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("T,K,N,L,r", CASES)
@pytest.mark.parametrize("swap", [False, True], ids=["as listed", "K and N changed"])
def test_the_formula_holds_for_weights_that_are_not_finite(T, K, N, L, r, bad, swap):
    if swap:
        K, N = N, K
    g = torch.Generator().manual_seed(T + K)
    inf = float("inf")
    ids = torch.randint(-1, L, (T,), generator=g)
    ids[:3] = torch.tensor([0, 1, -1])
    x, W = whole(g, (T, K), min(0.5, 12 / K)), whole(g, (N, K), min(0.3, 12 / K))
    A, B = whole(g, (L, r, K), min(0.3, 12 / K)), whole(g, (L, N, r), 2 / r)
    dy = whole(g, (T, N), min(0.5, 12 / N))
    x[:2, 3], x[:2, K - 1], dy[:2, 1] = 1, 1, 1
    # adapter 0: in both weights, at outputs and columns far apart
    B[0, 1, 2], A[0, 2, K - 1], B[0, N - 1, r - 1] = bad, -inf, bad
    # 1: a rank whose z is infinite and whose weight of an output is too
    A[1, 4, 3], B[1, 1, 4], B[1, N - 1, 4], B[1, 2, 4] = inf, inf, -inf, 3
    if L > 2:  # 2: finite z, and weights of one output in two ranks, which may lie in different parts of K
        B[2, 3, 1], B[2, 3, r - 2], A[2, r - 1, 5] = bad, bad, bad
    shape = lm.make_proj_shape(T, K, N, L, r)
    d = [t.bfloat16().cuda() for t in (x, W, A, B, dy)]
    i, ws = ids.int().cuda(), lm.alloc_proj_workspace(shape)
    y, z = torch.empty_like(d[4]), torch.empty((T, r), device="cuda")
    lm.moe_lora_proj_forward(shape, d[0], i, d[1], d[2], d[3], ws, y, z=z)
    z64 = own(x, A, ids)
    same(z, z64, "z")
    same(y, x @ W.T + own(z64, B, ids), "y")
    assert bool(y[ids == 1].isinf().any())
    dx, dA, dB = (torch.empty_like(t) for t in (d[0], d[2], d[3]))
    lm.moe_lora_proj_backward(shape, d[4], d[0], i, z, d[1], d[2], d[3], ws, dx=dx, dA=dA, dB=dB)
    u = own(dy, B.transpose(1, 2), ids)
    same(dx, dy @ W + own(u, A.transpose(1, 2), ids), "dx")
    for l in range(L):
        at = ids == l
        same(dA[l], u[at].T @ x[at], f"dA {l}")
        same(dB[l], dy[at].T @ z64[at], f"dB {l}")

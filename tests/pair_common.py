"""Inputs of whole numbers on which the gated block is exact up to 16 tokens:
every value that goes from one product to the next (h, dg, du) is a whole
number of up to 16 bits, which a sum of two bf16 holds and one bf16 does not,
the gates are saturated (act(g) = g, act' = 1 from g = 18 on), and all sums
stay below 2^24.  An output is then the exact whole number rounded once to
bf16, and every remainder that goes astray shows in its bits."""
from __future__ import annotations

import torch


def whole(shape, lo, hi, gen):
    """Whole numbers lo..hi in 64 bits."""
    return torch.randint(lo, hi + 1, shape, generator=gen).double()


def sign(shape, gen):
    return whole(shape, 0, 1, gen) * 2 - 1


def sparse(shape, per_sum, n, gen):
    """-1, 0, 1, about per_sum of a sum's n terms not zero."""
    return sign(shape, gen) * (torch.rand(shape, generator=gen) < min(1.0, per_sum / n))


def exact_product(a, b):
    """a b, with the sums of sizes checked to be exact in fp32."""
    assert float((a.abs() @ b.abs()).max()) < 2 ** 24
    return a @ b


def once(v):
    """Rounded to bf16, without a remainder."""
    return v.float().bfloat16().double()


def as_pair(v):
    """As the sum of two bf16."""
    hi = once(v)
    return hi + once(v - hi)


def forward_case(T, H, I, seed):
    """x, W_gu, W_down (64 bits, exact in bf16)."""
    g = torch.Generator().manual_seed(seed)
    cols = torch.randperm(H, generator=g)
    few = cols[2:14]
    x, W_gu = torch.zeros((T, H), dtype=torch.float64), torch.zeros((2 * I, H), dtype=torch.float64)
    x[:, cols[0]], x[:, cols[1]] = 1, 256
    W_gu[:I, cols[0]] = whole((I,), 64, 127, g)
    W_gu[I:, cols[1]] = sign((I,), g)
    x[:, few] = whole((T, len(few)), -2, 2, g)
    W_gu[:, few] = whole((2 * I, len(few)), -1, 1, g)
    return x, W_gu, sparse((H, I), 64, I, g)


def forward_exact(x, W_gu, W_down, carry=as_pair):
    """gu and y; carry: what becomes of h on its way."""
    I = W_down.shape[1]
    gu = exact_product(x, W_gu.T)
    assert float(gu[:, :I].min()) >= 18
    h = gu[:, :I] * gu[:, I:]
    assert float(h.abs().max()) < 2 ** 16
    return gu, exact_product(carry(h), W_down.T)


def backward_case(T, H, I, seed):
    """dy, x, gu, W_gu, W_down."""
    g = torch.Generator().manual_seed(seed)
    dy = torch.zeros((T, H), dtype=torch.float64)
    dy[:, torch.randperm(H, generator=g)[:4]] = whole((T, 4), -2, 2, g)
    dy[:, 0] = whole((T,), 1, 3, g)
    gu = torch.cat((whole((T, I), 64, 127, g), sign((T, I), g) * (2 * whole((T, I), 128, 254, g) + 1)), 1)
    return dy, whole((T, H), -3, 3, g), gu, sparse((2 * I, H), 128, 2 * I, g), whole((H, I), -1, 1, g)


def backward_exact(dy, x, gu, W_gu, W_down, carry=as_pair):
    I = W_down.shape[1]
    dh = exact_product(dy, W_down)
    h, dgu = gu[:, :I] * gu[:, I:], torch.cat((dh * gu[:, I:], dh * gu[:, :I]), 1)
    assert float(h.abs().max()) < 2 ** 16 and float(dgu.abs().max()) < 2 ** 16
    return dict(dx=exact_product(carry(dgu), W_gu), dW_gu=exact_product(carry(dgu).T, x),
                dW_down=exact_product(dy.T, carry(h)))


def w4_case(M, H, I, group, zeros, seed):
    """x (64 bits) and the three matrices' (q, scales, zero points), scales of
    one, with their values: h has up to 10 bits, so that the sums of h (128 +
    q) are exact too."""
    g = torch.Generator().manual_seed(seed)
    cols = torch.randperm(H, generator=g)
    few = cols[2:8]
    x = torch.zeros((M, H), dtype=torch.float64)
    x[:, cols[:2]] = 4
    x[:, few] = whole((M, len(few)), -1, 1, g)
    gate, up = (torch.zeros((I, H), dtype=torch.float64) for _ in range(2))
    gate[:, cols[0]] = whole((I,), 6, 7, g)
    gate[:, few] = whole((I, len(few)), -1, 0, g)
    up[:, cols[1]] = sign((I,), g) * whole((I,), 5, 6, g)
    up[:, few] = whole((I, len(few)), -1, 1, g)
    down = sparse((H, I), 64, I, g) * whole((H, I), 1, 2, g)

    def packed(v):
        n, k = v.shape
        G = (k + group - 1) // group
        z = whole((n, G), 7, 8, g) if zeros else torch.full((n, G), 8.0, dtype=torch.float64)
        q = (v + z[:, torch.arange(k) // group]).to(torch.uint8)
        assert int(q.max()) < 16
        return ((q[:, 0::2] | q[:, 1::2] << 4).contiguous(), torch.ones((n, G), dtype=torch.bfloat16),
                z.to(torch.uint8) if zeros else None)

    return x, [packed(v) for v in (gate, up, down)], (gate, up, down)


def w4_exact(x, values, carry=as_pair):
    gate, up, down = values
    g, u = exact_product(x, gate.T), exact_product(x, up.T)
    assert float(g.min()) >= 18
    h = g * u
    assert float(h.abs().max()) < 2 ** 10
    # 32 terms of h (128 + q) between two groups of zero points
    assert 32 * float(h.abs().max()) * (128 + 15) < 2 ** 24
    return exact_product(carry(h), down.T)


# rows of each form (up to 4, up to 8, one fragment), K short and split over
# the grid, one grid of gradients and three
FFN_CASES = [(1, 64, 64), (2, 264, 72), (4, 136, 1000), (5, 72, 328), (8, 512, 256), (9, 1000, 328), (15, 264, 1016),
             (16, 256, 4096), (16, 2056, 512), (13, 2056, 5512)]
W4_CASES = [(1, 264, 72, 32), (2, 64, 136, 128), (3, 1000, 264, 64), (8, 136, 520, 32), (9, 72, 1000, 64),
            (16, 512, 256, 128), (16, 128, 4096, 32), (8, 2560, 14336, 128)]

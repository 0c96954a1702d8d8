"""64-bit forms of the dense operators (on the CPU, from the bf16 inputs'
values), with bounds on what the kernels' roundings may do to each output.

Half a step of bf16 is 2^-8 of the value, of fp32 2^-24.  The bounds are worst
cases per element: every rounding at its full half step and all of one sign.
"""
from __future__ import annotations

import math

import torch

HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24
TINY = 1e-30
C2 = 2.0 * math.sqrt(2.0 / math.pi)


def act64(g, kind):
    """act(g) and its derivative in 64 bits."""
    if kind == "silu":
        p, dp = g, torch.ones_like(g)
    else:
        p, dp = C2 * (g + 0.044715 * g ** 3), C2 * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(p)
    return g * s, s + g * s * (1 - s) * dp


def ffn64(x, W_gu, W_down, act):
    I = W_down.shape[1]
    gu = x @ W_gu.T
    a, _ = act64(gu[:, :I], act)
    h = a * gu[:, I:]
    return gu, h, h @ W_down.T


# |act'| <= 1.13 for both gates and |act(g) - act(g')| <= 1.13 |g - g'|; the
# gate itself (exp, division, products) adds at most 32 fp32 half steps of
# |act(g)| + |g| * 2^-24 for the exponent's argument
LIP = 1.13


def ffn_bounds(x, W_gu, W_down, act):
    """64-bit (gu, h, y) and bounds on the kernels' errors in gu, h (before
    its rounding to bf16) and y."""
    I = W_down.shape[1]
    H = x.shape[1]
    gu, h, y = ffn64(x, W_gu, W_down, act)
    e_gu = (H + 4) * HALF_F32 * (x.abs() @ W_gu.abs().T)
    g, u = gu[:, :I], gu[:, I:]
    a, _ = act64(g, act)
    e_a = LIP * e_gu[:, :I] + 64 * HALF_F32 * (a.abs() + g.abs())
    e_h = e_a * u.abs() + (a.abs() + e_a) * e_gu[:, I:] + 2 * HALF_F32 * h.abs()
    e_hr = e_h + HALF_BF16 * (h.abs() + e_h)  # rounded
    e_y = e_hr @ W_down.abs().T + (I + 4) * HALF_F32 * ((h.abs() + e_hr) @ W_down.abs().T)
    e_y = e_y + HALF_BF16 * (y.abs() + e_y)
    return (gu, h, y), (e_gu, e_hr, e_y)


def ffn_backward_bounds(dy, x, gu, W_gu, W_down, act):
    """64-bit (dx, dW_gu, dW_down) from the kept gu, and bounds."""
    I = W_down.shape[1]
    T, H = x.shape
    g, u = gu[:, :I], gu[:, I:]
    a, da = act64(g, act)
    dh = dy @ W_down
    e_dh = (H + 4) * HALF_F32 * (dy.abs() @ W_down.abs())
    e_a = 64 * HALF_F32 * (a.abs() + g.abs())
    e_da = 256 * HALF_F32 * (1 + g.abs())
    h = a * u
    dg, du = dh * u * da, dh * a
    e_h = e_a * u.abs() + HALF_BF16 * h.abs() * 1.01
    e_dg = (e_dh * da.abs() + (dh.abs() + e_dh) * e_da) * u.abs() + HALF_BF16 * 1.01 * dg.abs()
    e_du = e_dh * a.abs() + (dh.abs() + e_dh) * e_a + HALF_BF16 * 1.01 * du.abs()
    dgu, e_dgu = torch.cat((dg, du), 1), 1.01 * torch.cat((e_dg, e_du), 1)

    def product(A, eA, B, eB, K):
        v = A @ B
        e = eA @ B.abs() + (A.abs() + eA) @ eB if eB is not None else eA @ B.abs()
        e = e + (K + 4) * HALF_F32 * ((A.abs() + eA) @ (B.abs() + (eB if eB is not None else 0)))
        return v, e + HALF_BF16 * (v.abs() + e)

    zero = torch.zeros_like
    return dict(dx=product(dgu, e_dgu, W_gu, None, 2 * I),
                dW_gu=product(dgu.T, e_dgu.T, x, None, T),
                dW_down=product(dy.T, zero(dy.T), h, e_h, T))


def within(got, want, bound, what):
    """Every element within its bound; its relative L2 error printed."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = (got - want).abs()
    worst = float((err / (bound + TINY)).max()) if err.numel() else 0.0
    l2 = float((got - want).norm() / max(float(want.norm()), TINY))
    print(f"[{what}] worst error / bound {worst:.3f}, relative L2 {l2:.2e}", flush=True)
    assert torch.isfinite(got).all() and worst <= 1.0, (what, worst)
    return l2


def ffn_inputs(T, H, I, seed, scale=1.0):
    """bf16 inputs on the CPU: x, W_gu, W_down, dy."""
    g = torch.Generator().manual_seed(seed)
    def rn(shape, std):
        return (torch.randn(shape, generator=g) * std).bfloat16()
    return (rn((T, H), scale), rn((2 * I, H), H ** -0.5), rn((H, I), I ** -0.5), rn((T, H), 1e-2))


def w4_inputs(N, K, group, zeros, seed):
    g = torch.Generator().manual_seed(seed)
    G = (K + group - 1) // group
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = ((0.5 + torch.rand((N, G), generator=g)) * 0.2 * K ** -0.5).bfloat16()
    z = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8) if zeros else None
    return q, s, z


def w4_values(q, s, z, group):
    """The weights in 64 bits, and the bound |w| + (128 + z) s that the
    kernel's summands have."""
    N, K = q.shape[0], 2 * q.shape[1]
    v = torch.empty((N, K), dtype=torch.float64)
    v[:, 0::2], v[:, 1::2] = (q & 15).double(), (q >> 4).double()
    col = torch.arange(K) // group
    zz = z.double()[:, col] if z is not None else torch.full((N, K), 8.0, dtype=torch.float64)
    ss = s.double()[:, col]
    return (v - zz) * ss, (2 * 128 + v + zz) * ss.abs()


def w4_bounds(x, w, mag):
    """y and its bound: fp32 sums of terms of size |x| mag, one rounding."""
    y = x @ w.T
    e = (x.shape[1] + 8) * HALF_F32 * (x.abs() @ mag.T)
    return y, e, e + HALF_BF16 * (y.abs() + e)

"""64-bit forms of the shared projection with adapters, with bounds on what the
kernels' roundings may do to each output.

Every fp32 sum of n terms is off by at most (n + 4) 2^-24 of the sum of their
sizes; s_l z and u go on as pairs of bf16, off by 2^-16 (the remainder, at most
2^-8 of the value, is rounded to half a step, 2^-8 of itself); results are
rounded to bf16 once, half a step, 2^-8."""
import torch

from dense_common import HALF_BF16, HALF_F32

PAIR = 2.0 ** -16


def inputs(T, K, N, L, r, seed, ids="each", scales=True):
    """x, W, A, B, dy (bf16), ids (int32), scales (fp32 or None), on the CPU."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda shape, std: (torch.randn(shape, generator=g) * std).bfloat16()  # noqa: E731
    x, W, A, B, dy = (rn((T, K), 1.0), rn((N, K), K ** -0.5), rn((L, r, K), K ** -0.5), rn((L, N, r), r ** -0.5),
                      rn((T, N), 1e-2))
    if ids == "each":
        i = torch.randint(0, L, (T,), generator=g)
    elif ids == "runs":
        cuts = torch.randint(0, T + 1, (max(1, T // 40),), generator=g).sort()[0]
        of = torch.randint(-1, L, (len(cuts) + 1,), generator=g)
        i = of[torch.searchsorted(cuts, torch.arange(T), right=True)]
    elif ids == "mixed":    # none, and ids that are no adapter's
        i = torch.randint(-1, L, (T,), generator=g)
        bad = torch.rand(T, generator=g)
        i = torch.where(bad < 0.1, L, torch.where(bad < 0.2, -7, torch.where(bad < 0.25, 2 ** 31 - 1, i)))
    elif ids == "none":
        i = torch.full((T,), -1)
    else:                   # one
        i = torch.full((T,), L - 1)
    s = (torch.rand(L, generator=g) * 3 - 1) if scales else None
    return x, W, A, B, dy, i.int(), s


def row_scale(ids, scales, lora_scale, L):
    """s_l of each token in 64 bits as the kernels form it (fp32), 0 without an
    adapter, and the adapter's index (0 there)."""
    has = (ids >= 0) & (ids < L)
    l = torch.where(has, ids, 0).long()
    s = torch.tensor(lora_scale, dtype=torch.float32, device=ids.device)
    s = (s * scales if scales is not None else s.repeat(L))[l]
    return torch.where(has, s.double(), 0.0), l, has


def _own(v, w, l, has):
    """w[l_t] v_t of every token with an adapter, one adapter after the other
    (zeros for the rest); w [L, out, in]."""
    out = v.new_zeros((v.shape[0], w.shape[1]))
    for a in range(w.shape[0]):
        at = torch.nonzero(has & (l == a)).flatten()
        if len(at):
            out[at] = v[at] @ w[a].T
    return out


def _down(v, w, s, l, has):
    """s (w v) of each token's own w [L, r, depth], its bound, and the product
    without s with its."""
    depth = w.shape[2]
    p = _own(v, w, l, has)
    e = (depth + 4) * HALF_F32 * _own(v.abs(), w.abs(), l, has)
    sp = s[:, None] * p
    e_sp = s.abs()[:, None] * e
    e_sp = e_sp + (PAIR + 4 * HALF_F32) * (sp.abs() + e_sp)
    return p, e, sp, e_sp


def _join(v, w, sp, e_sp, back, l, has):
    """v w^T + back sp with each token's own back [L, out, r], and the bound,
    before the rounding to bf16."""
    depth, r = v.shape[1], sp.shape[1]
    y = v @ w.T + _own(sp, back, l, has)
    off = _own(e_sp, back.abs(), l, has)
    size = v.abs() @ w.abs().T + _own(sp.abs(), back.abs(), l, has) + off
    return y, (depth + 2 * r + 8) * HALF_F32 * size + off


def rounded(v, e):
    return v, e + HALF_BF16 * (v.abs() + e)


def forward64(x, W, A, B, ids, scales, lora_scale=1.0):
    """(z, bound), (y, bound); everything in 64 bits."""
    s, l, has = row_scale(ids, scales, lora_scale, A.shape[0])
    z, e_z, sz, e_sz = _down(x, A, s, l, has)
    return (z, e_z), rounded(*_join(x, W, sz, e_sz, B, l, has))


def backward64(dy, x, z, W, A, B, ids, scales, lora_scale=1.0):
    """dx, dA and dB with their bounds, from the kept z."""
    L, r, K = A.shape
    N = W.shape[0]
    s, l, has = row_scale(ids, scales, lora_scale, L)
    _, _, u, e_u = _down(dy, B.transpose(1, 2), s, l, has)
    dx = rounded(*_join(dy, W.T, u, e_u, A.transpose(1, 2), l, has))
    sz = s[:, None] * z
    e_sz = (PAIR + 4 * HALF_F32) * sz.abs()
    dA, eA, dB, eB = (x.new_zeros(n) for n in ((L, r, K), (L, r, K), (L, N, r), (L, N, r)))
    for a in range(L):
        at = torch.nonzero(has & (l == a)).flatten()
        n = 2 * len(at) + 16  # pairs, and the slabs' additions
        dA[a] = u[at].T @ x[at]
        eA[a] = e_u[at].T @ x[at].abs() + n * HALF_F32 * ((u[at].abs() + e_u[at]).T @ x[at].abs())
        dB[a] = dy[at].T @ sz[at]
        eB[a] = dy[at].abs().T @ e_sz[at] + n * HALF_F32 * (dy[at].abs().T @ (sz[at].abs() + e_sz[at]))
    return dict(dx=dx, dA=rounded(dA, eA), dB=rounded(dB, eB))

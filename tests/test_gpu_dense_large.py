"""The dense operators at their largest: offsets past 2^31, many rows of 4-bit
products, K splits with several row tiles."""
import pytest
import torch

from dense_common import (HALF_BF16, act64, ffn_backward_bounds, ffn_bounds, ffn_inputs, w4_bounds, w4_inputs, w4_values,
                          within)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [(200, 64, 4096, 128), (1000, 300, 2056, 64), (4097, 40, 1032, 32),
                                         (65536, 17, 72, 32)])
def test_many_rows(M, N, K, group, zeros):
    import lora_moe_amd as lm
    parts = w4_inputs(N, K, group, zeros, N + K)
    w = lm.moe_lora_w4_pack(*(None if t is None else t.cuda() for t in parts), group=group)
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).bfloat16()
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_w4_matmul(x.cuda(), w, y)
    want, _, bound = w4_bounds(x.double(), *w4_values(*parts, group))
    within(y, want, bound, f"M={M} N={N} K={K} group={group}")


@pytest.mark.parametrize("M", [2, 20])
def test_packed_weights_past_two_gigabytes(M):
    import lora_moe_amd as lm
    N, K, group = (1 << 18) + 5, (1 << 14) + 8, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
    s = ((0.5 + torch.rand((N, (K + group - 1) // group), generator=gen, device="cuda")) * 1e-3).bfloat16()
    w = lm.moe_lora_w4_pack(q, s, group=group)
    assert w.packed.numel() > 2 ** 31
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).bfloat16()
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_w4_matmul(x.cuda(), w, y)
    border = 2 ** 31 // (K // 2)
    n = torch.tensor([0, 1, 15, 16, 100000, *range(border - 40, border + 40), N - 17, N - 6, N - 2, N - 1])
    want, _, bound = w4_bounds(x.double(), *w4_values(q[n.cuda()].cpu(), s[n.cuda()].cpu(), None, group))
    within(y[:, n.cuda()], want, bound, f"M={M}, {w.packed.numel()} bytes")


def test_block_with_more_than_two_to_the_31_values():
    """2.3e9 kept pre-activations (9 GB), 1.1e9 values of h: rows from both
    ends and around 2^31, and the weights' gradients."""
    import lora_moe_amd as lm
    T, H, I = 140001, 8, 8200
    x, W_gu, W_down, dy = ffn_inputs(T, H, I, 12)
    xd, gd, dd, dyd = (t.cuda() for t in (x, W_gu, W_down, dy))
    shape = lm.make_ffn_shape(T, H, I)
    ws = lm.alloc_ffn_workspace(shape)
    y, dx, dW_gu, dW_down = (torch.full_like(t, float("nan")) for t in (xd, xd, gd, dd))
    gu = torch.full((T, 2 * I), float("nan"), device="cuda")
    assert gu.numel() > 2 ** 31
    lm.moe_lora_ffn_forward(shape, xd, gd, dd, ws, y, gu=gu)
    lm.moe_lora_ffn_backward(shape, dyd, xd, gu, gd, dd, ws, dx=dx, dW_gu=dW_gu, dW_down=dW_down)
    border = 2 ** 31 // (2 * I)
    rows = torch.tensor([0, 1, 2 ** 16, *range(border - 2, border + 3), T - 2, T - 1])
    (gu64, _, y64), (e_gu, _, e_y) = ffn_bounds(x[rows].double(), W_gu.double(), W_down.double(), "silu")
    within(gu[rows.cuda()], gu64, e_gu, "gu")
    within(y[rows.cuda()], y64, e_y, "y")
    kept = gu[rows.cuda()].double().cpu()
    v, e = ffn_backward_bounds(dy[rows].double(), x[rows].double(), kept, W_gu.double(), W_down.double(), "silu")["dx"]
    within(dx[rows.cuda()], v, e, "dx")
    # the sums over the tokens, in 64 bits on the GPU, a few thousand tokens at a time
    want = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (gd, dd)]
    for t0 in range(0, T, 8192):
        part = slice(t0, min(t0 + 8192, T))
        g, u = gu[part, :I].double(), gu[part, I:].double()
        a, da = act64(g, "silu")
        dh = dyd[part].double() @ dd.double()
        want[0] += torch.cat((dh * u * da, dh * a), 1).T.contiguous() @ xd[part].double()
        want[1] += dyd[part].double().T.contiguous() @ (a * u)
    for got, w in zip((dW_gu, dW_down), want):
        # two independent roundings to bf16, each 2^-8 / sqrt(3) in the mean square at most, 1.3 for the spread
        l2 = float((got.double() - w).norm() / w.norm())
        print(f"relative L2 {l2:.2e}", flush=True)
        assert l2 <= 1.3 * HALF_BF16 * (2 / 3) ** 0.5

"""Up to 16 tokens h, dg and du go from one product to the next as sums of
two bf16: on whole numbers every output is exact."""
import pytest
import torch

import pair_common as pc

pytestmark = pytest.mark.gpu


def same(got, want, what):
    """Bit for bit the exact whole numbers rounded once."""
    want = want.float().bfloat16()
    bad = int((got.cpu() != want).sum())
    print(f"[{what}] {bad} of {want.numel()} differ", flush=True)
    assert bad == 0, (what, bad)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", pc.FFN_CASES)
def test_block(T, H, I, act):
    import lora_moe_amd as lm
    shape = lm.make_ffn_shape(T, H, I, act)
    ws = lm.alloc_ffn_workspace(shape)
    what = f"T={T} H={H} I={I} {act}"
    case = pc.forward_case(T, H, I, T + H)
    gu64, y64 = pc.forward_exact(*case)
    dev = [t.bfloat16().cuda() for t in case]
    y, gu = torch.empty_like(dev[0]), torch.empty((T, 2 * I), device="cuda")
    for kept in (gu, None):
        lm.moe_lora_ffn_forward(shape, *dev, ws, y.fill_(float("nan")), gu=kept)
        same(y, y64, what + " y")
    assert torch.equal(gu.double().cpu(), gu64)
    case = pc.backward_case(T, H, I, T + I)
    want = pc.backward_exact(*case)
    dy, x, gu, W_gu, W_down = (t.float().cuda() if i == 2 else t.bfloat16().cuda() for i, t in enumerate(case))
    like = dict(dx=x, dW_gu=W_gu, dW_down=W_down)
    for names in (list(want), *([n] for n in want)):  # one grid where sizes are small, and each by itself
        out = {n: torch.full_like(like[n], float("nan")) for n in names}
        lm.moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, ws, **out)
        for n in names:
            same(out[n], want[n], f"{what} {n} of {len(names)}")


@pytest.mark.parametrize("act,zeros", [("silu", False), ("gelu", True)])
@pytest.mark.parametrize("M,H,I,group", pc.W4_CASES)
def test_4_bit_block(M, H, I, group, act, zeros):
    import lora_moe_amd as lm
    x, parts, values = pc.w4_case(M, H, I, group, zeros, M + I)
    w = [lm.moe_lora_w4_pack(*(None if t is None else t.cuda() for t in p), group=group) for p in parts]
    y = torch.full((M, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.moe_lora_w4_ffn_forward(x.bfloat16().cuda(), *w, lm.alloc_w4_ffn_workspace(M, I), y, act=act)
    same(y, pc.w4_exact(x, values), f"M={M} H={H} I={I} group={group} {act}")

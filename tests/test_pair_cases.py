"""The whole-number cases are what they claim: sums of two bf16 give the
exact outputs, and a block that loses its remainders gives others."""
import pytest
import torch

import pair_common as pc


def differ(a, b):
    return int((a.float().bfloat16() != b.float().bfloat16()).sum())


@pytest.mark.parametrize("T,H,I", pc.FFN_CASES)
def test_block_shows_lost_remainders(T, H, I):
    case = pc.forward_case(T, H, I, T + H)
    exact, lost = (pc.forward_exact(*case, carry=c)[1] for c in (lambda v: v, pc.once))
    assert torch.equal(pc.forward_exact(*case)[1], exact)
    assert differ(exact, lost) > exact.numel() // 10
    case = pc.backward_case(T, H, I, T + I)
    exact, pair, lost = (pc.backward_exact(*case, carry=c) for c in (lambda v: v, pc.as_pair, pc.once))
    for n in exact:
        assert torch.equal(pair[n], exact[n]), n
        # (a single token's h or dgu is alone in its sum: times a power of two it is rounded alike either way)
        assert differ(exact[n], lost[n]) > 0 or (T == 1 and n != "dx"), n


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,H,I,group", pc.W4_CASES)
def test_4_bit_block_shows_lost_remainders(M, H, I, group, zeros):
    x, _, values = pc.w4_case(M, H, I, group, zeros, M + I)
    exact, pair, lost = (pc.w4_exact(x, values, c) for c in (lambda v: v, pc.as_pair, pc.once))
    assert torch.equal(pair, exact) and differ(exact, lost) > exact.numel() // 20

"""How the binding looks at its tensors on the GPU: views, leaves of autograd,
sizes of one, and what is refused there."""
import pytest
import torch

import lora_moe_amd as lm

pytestmark = pytest.mark.gpu


def whole(*sizes, seed=0):
    """Small whole numbers, whose sums are exact in any order."""
    g = torch.Generator().manual_seed(seed + sum(sizes))
    return torch.randint(-2, 3, sizes, generator=g).to(torch.bfloat16).cuda()


def test_views_and_leaves_are_operands():
    T, K, N, L, r = 5, 72, 40, 3, 8
    x, W, A, B = whole(T + 2, K), whole(N + 1, K), whole(L, r, K), whole(L + 1, N, r)
    ids = torch.tensor([9, 9, 9, 9, 0, 2, -1, 1, 2], dtype=torch.int32, device="cuda")
    want = lm.lora_projection(x[2:].clone(), ids[4:].clone(), W[1:].clone(), A, B[1:].clone())
    ref = x[2:].double() @ W[1:].double().t()
    for t, l in enumerate([0, 2, -1, 1, 2]):
        if l >= 0:
            ref[t] += (x[2 + t].double() @ A[l].double().t()) @ B[1 + l].double().t()
    assert torch.equal(want, ref.to(torch.bfloat16))
    # views that begin inside their storage (16-byte aligned), and leaves
    leaves = [t.clone().requires_grad_() for t in (x, W, A, B)]
    y = lm.lora_projection(leaves[0][2:], ids[4:], leaves[1][1:], leaves[2], leaves[3][1:])
    assert torch.equal(y, want) and not y.requires_grad
    y = lm.lora_projection(leaves[0].detach()[2:], ids[4:], leaves[1][1:], torch.nn.Parameter(A), B[1:])
    assert torch.equal(y, want)
    # strides of sizes of one and of empty tensors say nothing
    one = x[:1].as_strided((1, K), (7, 1))
    assert torch.equal(lm.lora_projection(one, ids[:1], W[:N], A, B[:L]), x[:1] @ W[:N].t())
    empty = x[:0].as_strided((0, K), (1, 5))
    assert lm.lora_projection(empty, ids[:0], W[:N], A, B[:L]).shape == (0, N)


@pytest.mark.parametrize("change,match", [
    (dict(x=lambda t: t.t().contiguous().t()), "x must be contiguous"),
    (dict(x=lambda t: t.float()), "x: dtype float32, expected bfloat16"),
    (dict(x=lambda t: t.cpu()), "device tensors"),
    (dict(ids=lambda t: t.long()), "lora_ids: dtype int64, expected int32"),
    (dict(ids=lambda t: t[:4]), r"lora_ids: shape \(4,\), expected \(5,\)"),
    (dict(B=lambda t: t[:, :, :4].contiguous()), "B: shape"),
    (dict(A=lambda t: t.cpu()), r"device tensors \(A is on cpu\)")])
def test_refusals_name_the_operand(change, match):
    T, K, N, L, r = 5, 72, 40, 3, 8
    ops = dict(x=whole(T, K), ids=torch.zeros(T, dtype=torch.int32, device="cuda"), W=whole(N, K), A=whole(L, r, K),
               B=whole(L, N, r))
    s = lm.make_proj_shape(T, K, N, L, r)
    ws, y = lm.alloc_proj_workspace(s), torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for k, f in change.items():
        ops[k] = f(ops[k])
    with pytest.raises(ValueError, match=match):
        lm.moe_lora_proj_forward(s, ops["x"], ops["ids"], ops["W"], ops["A"], ops["B"], ws, y)
    torch.cuda.synchronize()
    assert bool((y == 7).all())


def test_a_view_that_is_not_aligned_is_refused():
    T, K, N, L, r = 5, 72, 40, 3, 8
    flat = whole(T * K + 1)
    s = lm.make_proj_shape(T, K, N, L, r)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    args = [torch.zeros(T, dtype=torch.int32, device="cuda"), whole(N, K), whole(L, r, K), whole(L, N, r)]
    with pytest.raises(lm.MoeLoraError):
        lm.moe_lora_proj_forward(s, flat[1:].view(T, K), *args, lm.alloc_proj_workspace(s), y)
    with pytest.raises(ValueError, match="workspace holds"):
        lm.moe_lora_proj_forward(s, flat[:-1].view(T, K), *args, torch.empty(8, dtype=torch.uint8, device="cuda"), y)
    torch.cuda.synchronize()
    assert bool((y == 7).all())

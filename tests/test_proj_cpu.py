"""The shared projection with adapters: host-side checks (each refusal returns
its code, or raises, without touching a GPU), the bounds' 64-bit forms, and
what the compiler puts before the copies' assembly."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import lora_moe_amd as lm
from proj_common import backward64, forward64, inputs

OK, EINVAL, EALIGN, EWS, EUNSUP = (lm.MOE_LORA_OK, lm.MOE_LORA_EINVAL, lm.MOE_LORA_EALIGN, lm.MOE_LORA_EWORKSPACE,
                                   lm.MOE_LORA_EUNSUPPORTED)
BASE, STEP = 1 << 40, 1 << 38  # addresses far apart that nothing ever reads
FORWARD = ("x", "lora_ids", "W", "A", "B", "scales", "z", "ws", "n", "y")
BACKWARD = ("dy", "x", "lora_ids", "z", "W", "A", "B", "scales", "ws", "n", "dx", "dA", "dB")


def at(i, off=0):
    return BASE + i * STEP + off


@pytest.fixture(scope="module")
def lib():
    return lm.load_library()


def forward(lib, s, **over):
    a = dict({n: at(i) for i, n in enumerate(FORWARD)}, n=1 << 34)
    a.update(over)
    return lib.moe_lora_proj_forward(ctypes.byref(s) if s else None, *[a[n] for n in FORWARD], None)


def backward(lib, s, **over):
    a = dict({n: at(i) for i, n in enumerate(BACKWARD)}, n=1 << 34)
    a.update(over)
    return lib.moe_lora_proj_backward(ctypes.byref(s) if s else None, *[a[n] for n in BACKWARD], None)


@pytest.mark.parametrize("sizes,code", [
    ((-1, 64, 64, 2, 8), EINVAL), ((4, 0, 64, 2, 8), EINVAL), ((4, 64, -8, 2, 8), EINVAL), ((4, 64, 64, 0, 8), EINVAL),
    ((4, 64, 64, 2, 0), EINVAL), ((4, 60, 64, 2, 8), EALIGN), ((4, 64, 68, 2, 8), EALIGN), ((4, 64, 64, 2, 12), EUNSUP),
    ((4, 64, 64, 2, 136), EUNSUP), ((4, 64, 64, 2048, 8), EUNSUP), (((1 << 17) + 1, 8, 8, 1, 8), EUNSUP),
    ((4, (1 << 20) + 8, 8, 1, 8), EUNSUP), ((4, 8, (1 << 20) + 8, 1, 8), EUNSUP),
    # x, y, A and B of 2 GiB
    ((1 << 17, 8192, 8, 1, 8), EUNSUP), ((1 << 17, 8, 8192, 1, 8), EUNSUP), ((4, 8192, 8, 1024, 128), EUNSUP),
    ((4, 8, 8192, 1024, 128), EUNSUP)])
def test_proj_shapes(lib, sizes, code):
    s = lm.moe_lora_proj_shape(*sizes, 1.0)
    assert forward(lib, s) == code and backward(lib, s) == code
    assert lm.moe_lora_proj_workspace_bytes(s) == 0
    with pytest.raises(lm.MoeLoraError):
        lm.alloc_proj_workspace(s, device="cpu")


@pytest.mark.parametrize("T", [4, 500])
def test_proj_arguments(lib, T):
    s = lm.make_proj_shape(T, 64, 128, 3, 16)
    assert forward(lib, None) == EINVAL and backward(lib, None) == EINVAL
    for n in ("x", "lora_ids", "W", "A", "B", "y"):
        assert forward(lib, s, **{n: None}) == EINVAL, n
    for n in ("dy", "x", "lora_ids", "z", "W", "A", "B"):
        assert backward(lib, s, **{n: None}) == EINVAL, n
    assert backward(lib, s, dx=None, dA=None, dB=None) == EINVAL
    for call, back in ((forward, False), (backward, True)):
        need = lm.moe_lora_proj_workspace_bytes(s, back)
        assert call(lib, s, ws=None) == EWS and call(lib, s, n=need - 1) == EWS
    for call, names in ((forward, FORWARD), (backward, BACKWARD)):
        for n in names:
            if n != "n":
                assert call(lib, s, **{n: at(20, 8)}) == EALIGN, n


def test_proj_overlaps(lib):
    """An output or the workspace on an input or another output, by its first
    or last bytes."""
    s = lm.make_proj_shape(40, 64, 128, 3, 16)
    f, b = FORWARD.index, BACKWARD.index
    for out, other, off in (("y", "x", 40 * 64 * 2 - 16), ("y", "W", 0), ("z", "scales", 0), ("z", "y", 32),
                            ("ws", "lora_ids", 144), ("ws", "B", 0), ("y", "A", 3 * 16 * 64 * 2 - 16)):
        assert forward(lib, s, **{out: at(f(other), off)}) == EINVAL, (out, other)
    for out, other, off in (("dx", "x", 0), ("dx", "dy", 16), ("dA", "A", 0), ("dB", "B", 3 * 128 * 16 * 2 - 16),
                            ("dB", "dA", 0), ("ws", "z", 0), ("dA", "dx", 64), ("ws", "dB", 0), ("dx", "lora_ids", 0)):
        assert backward(lib, s, **{out: at(b(other), off)}) == EINVAL, (out, other)


def test_proj_no_tokens(lib):
    s = lm.make_proj_shape(0, 64, 128, 3, 16)
    assert lm.moe_lora_proj_workspace_bytes(s) > 0
    assert forward(lib, s, **{n: None for n in FORWARD if n != "n"}) == OK
    assert backward(lib, s, **{n: None for n in BACKWARD if n != "n"}) == OK
    assert backward(lib, s, dA=at(BACKWARD.index("B"))) == EINVAL


def test_proj_binding():
    s = lm.make_proj_shape(2, 16, 24, 3, 8)
    z = lambda *d, t=torch.bfloat16: torch.zeros(d, dtype=t)  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    ws = z(lm.moe_lora_proj_workspace_bytes(s), t=torch.uint8)
    good = dict(x=z(2, 16), lora_ids=z(2, t=i32), W=z(24, 16), A=z(3, 8, 16), B=z(3, 24, 8), workspace=ws, y=z(2, 24))
    for over, text in ((dict(), "device tensors"), (dict(x=z(2, 16, t=torch.float16)), "dtype"),
                       (dict(lora_ids=z(2, t=torch.int64)), "dtype"), (dict(W=z(16, 24)), "shape"),
                       (dict(A=z(3, 16, 8).transpose(1, 2)), "contiguous"), (dict(B=z(2, 24, 8)), "shape"),
                       (dict(y=None), "required"), (dict(workspace=None), "required"), (dict(workspace=ws[:8]), "holds"),
                       (dict(z=z(2, 8)), "dtype"), (dict(scales=z(2, t=f32)), "shape")):
        with pytest.raises(ValueError, match=text):
            lm.moe_lora_proj_forward(s, **dict(good, **over))
    back = dict(dy=z(2, 24), x=z(2, 16), lora_ids=z(2, t=i32), z=z(2, 8, t=f32), W=z(24, 16), A=z(3, 8, 16),
                B=z(3, 24, 8), workspace=ws, dx=z(2, 16))
    for over, text in ((dict(), "device tensors"), (dict(dA=z(3, 16, 8)), "shape"), (dict(dB=z(3, 24, 8, t=f32)), "dtype"),
                       (dict(z=None), "required")):
        with pytest.raises(ValueError, match=text):
            lm.moe_lora_proj_backward(s, **dict(back, **over))
    with pytest.raises(ValueError, match="dimensions"):
        lm.lora_projection(z(2, 2, 16), z(2, t=i32), z(24, 16), z(3, 8, 16), z(3, 24, 8))
    with pytest.raises(ValueError, match="dimensions"):
        lm.lora_projection(z(2, 16), z(2, t=i32), z(24, 16), z(8, 16), z(3, 24, 8))


def test_the_64_bit_forms():
    """proj_common's gradients are those of its forward, by autograd."""
    T, K, N, L, r = 50, 24, 40, 5, 8
    x, W, A, B, dy, ids, s = inputs(T, K, N, L, r, 1, "mixed")
    f = [t.double() for t in (x, W, A, B, dy)]
    (z, _), (y, _) = forward64(*f[:4], ids, s, 0.5)
    leaves = [f[0].clone().requires_grad_(), f[2].clone().requires_grad_(), f[3].clone().requires_grad_()]
    rows = []
    for t, l in enumerate(ids.tolist()):
        row = f[1] @ leaves[0][t]
        if 0 <= l < L:
            row = row + (0.5 * s[l]).double() * (leaves[2][l] @ (leaves[1][l] @ leaves[0][t]))
        rows.append(row)
    out = torch.stack(rows)
    assert float((out - y).abs().max()) < 1e-12
    want = backward64(f[4], f[0], z, *f[1:4], ids, s, 0.5)
    for n, g in zip(("dx", "dA", "dB"), torch.autograd.grad(out, leaves, f[4])):
        assert float((want[n][0] - g).abs().max()) < 1e-12, n


@pytest.mark.parametrize("name,least", [("proj_gemm.hip", 200), ("proj_grads.hip", 40)])
def test_copies_keep_their_distance_from_vector_writes(tmp_path, name, least):
    """A vector instruction that writes a scalar register needs five wait
    states before a memory instruction that reads it; the compiler does not
    see into the copies' assembly, so what it puts before them is checked."""
    from lora_moe_amd import build
    out = str(tmp_path / "out.s")
    subprocess.run([build.HIPCC, *build.FLAGS, "-w", "-S", "--cuda-device-only", os.path.join(lm.PKG, "csrc", name),
                    "-o", out], check=True, capture_output=True)

    def scalars(text):
        regs = {int(n) for n in re.findall(r"\bs(\d+)\b", text)}
        for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
            regs |= set(range(int(a), int(b) + 1))
        return regs

    before, copies = [], 0
    with open(out) as f:
        for line in f:
            ins = line.split(";")[0].strip()
            if not ins or ins.startswith(".") or ins.endswith(":"):
                continue
            if ins.startswith("buffer_load") and ins.endswith(" lds"):
                copies += 1
                for w in before:
                    if w.startswith("v_") and not w.startswith("v_mfma"):
                        written = ",".join(w.split(",")[:2 if "_co_" in w else 1])
                        assert not scalars(written) & scalars(ins), (w, ins)
            before = before[-4:] + [ins]
    assert copies > least

"""The dense operators' host-side checks: each refusal returns its code, or
raises, without touching a GPU."""
import ctypes

import pytest
import torch

import lora_moe_amd as lm

EINVAL, EALIGN, EWS, EUNSUP = (lm.MOE_LORA_EINVAL, lm.MOE_LORA_EALIGN, lm.MOE_LORA_EWORKSPACE,
                               lm.MOE_LORA_EUNSUPPORTED)
# addresses far apart that nothing ever reads: every call here is refused
BASE, STEP = 1 << 40, 1 << 36


def at(i, off=0):
    return BASE + i * STEP + off


@pytest.fixture(scope="module")
def lib():
    return lm.load_library()


def ffn_forward(lib, s, **over):
    a = dict(x=at(0), W_gu=at(1), W_down=at(2), gu=at(3), ws=at(4), n=1 << 30, y=at(5))
    a.update(over)
    return lib.moe_lora_ffn_forward(ctypes.byref(s) if s else None, a["x"], a["W_gu"], a["W_down"], a["gu"],
                                    a["ws"], a["n"], a["y"], None)


def ffn_backward(lib, s, **over):
    a = dict(dy=at(0), x=at(1), gu=at(2), W_gu=at(3), W_down=at(4), ws=at(5), n=1 << 30, dx=at(6), dW_gu=at(7),
             dW_down=at(8))
    a.update(over)
    return lib.moe_lora_ffn_backward(ctypes.byref(s) if s else None, a["dy"], a["x"], a["gu"], a["W_gu"],
                                     a["W_down"], a["ws"], a["n"], a["dx"], a["dW_gu"], a["dW_down"], None)


@pytest.mark.parametrize("sizes,code", [
    ((-1, 64, 64, 0), EINVAL), ((4, 0, 64, 0), EINVAL), ((4, 64, -8, 0), EINVAL), ((4, 64, 64, 2), EINVAL),
    ((4, 64, 64, -1), EINVAL), ((4, 60, 64, 0), EALIGN), ((4, 64, 68, 1), EALIGN),
    ((4, (1 << 20) + 8, 64, 0), EUNSUP), ((4, 64, (1 << 20) + 8, 0), EUNSUP), (((1 << 26) + 1, 8, 8, 0), EUNSUP)])
def test_ffn_shapes(lib, sizes, code):
    s = lm.moe_lora_ffn_shape(*sizes)
    assert ffn_forward(lib, s) == code
    assert ffn_backward(lib, s) == code
    assert lm.moe_lora_ffn_workspace_bytes(s) == 0
    with pytest.raises(lm.MoeLoraError):
        lm.alloc_ffn_workspace(s, device="cpu")


def test_ffn_arguments(lib):
    s = lm.make_ffn_shape(4, 64, 128)
    assert ffn_forward(lib, None) == EINVAL and ffn_backward(lib, None) == EINVAL
    for n in ("x", "W_gu", "W_down", "y"):
        assert ffn_forward(lib, s, **{n: None}) == EINVAL, n
    for n in ("dy", "x", "gu", "W_gu", "W_down"):
        assert ffn_backward(lib, s, **{n: None}) == EINVAL, n
    assert ffn_backward(lib, s, dx=None, dW_gu=None, dW_down=None) == EINVAL
    for call, back in ((ffn_forward, False), (ffn_backward, True)):
        need = lm.moe_lora_ffn_workspace_bytes(s, back)
        assert call(lib, s, ws=None) == EWS
        assert call(lib, s, n=need - 1) == EWS
        assert call(lib, s, ws=at(5, 8)) == EALIGN
    for n in ("x", "W_gu", "W_down", "gu", "y"):
        assert ffn_forward(lib, s, **{n: at(9, 8)}) == EALIGN, n
    for n in ("dy", "x", "gu", "W_gu", "W_down", "dx", "dW_gu", "dW_down"):
        assert ffn_backward(lib, s, **{n: at(9, 4)}) == EALIGN, n


def test_ffn_no_tokens_backward(lib):
    s = lm.make_ffn_shape(0, 64, 128)
    assert ffn_backward(lib, s, dx=None, dW_gu=None, dW_down=None) == 0


def test_workspace_is_required():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace is required"):
        lm.moe_lora_ffn_forward(lm.make_ffn_shape(2, 64, 64), x, x, x, None, x)


def test_ffn_overlaps(lib):
    """An output or the workspace on an input or on another output, by its
    first or last 16 bytes."""
    s = lm.make_ffn_shape(4, 64, 128)
    last = 4 * 64 * 2 - 16
    assert ffn_forward(lib, s, y=at(0)) == EINVAL
    assert ffn_forward(lib, s, y=at(0, last)) == EINVAL
    assert ffn_forward(lib, s, ws=at(1)) == EINVAL
    assert ffn_forward(lib, s, gu=at(5, last)) == EINVAL
    assert ffn_backward(lib, s, dx=at(0)) == EINVAL
    assert ffn_backward(lib, s, dx=at(1, last)) == EINVAL
    assert ffn_backward(lib, s, dW_gu=at(3)) == EINVAL
    assert ffn_backward(lib, s, dW_gu=at(8)) == EINVAL
    assert ffn_backward(lib, s, ws=at(2)) == EINVAL


def test_ffn_no_tokens_forward(lib):
    s = lm.make_ffn_shape(0, 64, 128)
    assert lm.moe_lora_ffn_workspace_bytes(s) > 0
    assert ffn_forward(lib, s, x=None, y=None, gu=None, ws=None, n=0) == lm.MOE_LORA_OK


def test_ffn_binding():
    with pytest.raises(ValueError, match="act"):
        lm.make_ffn_shape(1, 8, 8, act="relu")
    s = lm.make_ffn_shape(2, 16, 8)
    z = lambda *d, t=torch.bfloat16: torch.zeros(d, dtype=t)  # noqa: E731
    ws = z(lm.moe_lora_ffn_workspace_bytes(s), t=torch.uint8)
    good = dict(x=z(2, 16), W_gu=z(16, 16), W_down=z(16, 8), workspace=ws, y=z(2, 16))
    for over, text in ((dict(), "device tensors"), (dict(x=z(2, 16, t=torch.float16)), "dtype"),
                       (dict(W_gu=z(8, 16)), "shape"), (dict(W_down=z(8, 16).t()), "contiguous"),
                       (dict(y=None), "required"), (dict(workspace=ws[:4]), "workspace"),
                       (dict(workspace=ws.view(1, -1)), "workspace"), (dict(gu=z(2, 16)), "dtype")):
        with pytest.raises(ValueError, match=text):
            lm.moe_lora_ffn_forward(s, **dict(good, **over))
    with pytest.raises(ValueError, match="shape"):
        lm.moe_lora_ffn_backward(s, z(2, 16), z(2, 16), z(2, 16, t=torch.float32), z(16, 16), z(16, 8), ws,
                                 dx=z(3, 16))
    with pytest.raises(ValueError, match="dimensions"):
        lm.gated_ffn(z(2, 2, 16), z(16, 16), z(16, 8))


def w4(N=32, K=64, group=32, zeros=0, data=at(0)):
    return lm.moe_lora_w4(data, N, K, group, zeros)


def w4_bytes(lib, d):
    return lib.moe_lora_w4_bytes(ctypes.byref(d))


def test_w4_matrices(lib):
    for d, code in ((w4(N=0), EINVAL), (w4(K=-8), EINVAL), (w4(group=16), EINVAL), (w4(group=0), EINVAL),
                    (w4(zeros=2), EINVAL), (w4(K=60), EALIGN), (w4(N=(1 << 22) + 1), EUNSUP),
                    (w4(K=(1 << 22) + 8), EUNSUP)):
        assert w4_bytes(lib, d) == 0
        assert lib.moe_lora_w4_matmul(ctypes.byref(d), 1, at(1), None, 0, at(2), None) == code
        z = at(4) if d.has_zeros else None
        assert lib.moe_lora_w4_pack(ctypes.byref(d), at(1), at(2), z, at(3), 1 << 40, None) == code
    # at least the weights, the scales and the zero points of whole tiles
    assert w4_bytes(lib, w4(17, 136, 32)) >= 32 * 256 // 2 + 32 * 5 * 2
    assert w4_bytes(lib, w4(17, 136, 32, 1)) >= w4_bytes(lib, w4(17, 136, 32)) + 32 * 5
    assert lib.moe_lora_w4_matmul(None, 1, at(1), None, 0, at(2), None) == EINVAL


def test_w4_arguments(lib):
    d, dz = w4(), w4(zeros=1)
    n = w4_bytes(lib, d)
    mm = lambda M=2, x=at(1), y=at(2), d=d, ws=at(9), n=1 << 30: lib.moe_lora_w4_matmul(  # noqa: E731
        ctypes.byref(d), M, x, ws, n, y, None)
    big = w4(128, 4096, 32)  # rows enough to split K
    need = lib.moe_lora_w4_workspace_bytes(ctypes.byref(big), 32)
    assert need > 256
    assert mm(M=32, d=big, n=need - 256) == EWS and mm(M=32, d=big, ws=None) == EWS
    assert mm(M=32, d=big, ws=at(9, 8)) == EALIGN and mm(M=32, d=big, ws=at(1)) == EINVAL
    assert mm(M=32, d=big, ws=at(2)) == EINVAL
    assert lib.moe_lora_w4_workspace_bytes(ctypes.byref(w4(K=60)), 1) == 0
    assert lib.moe_lora_w4_workspace_bytes(ctypes.byref(d), -1) == 0
    assert mm(M=-1) == EINVAL and mm(M=65537) == EUNSUP and mm(M=0, x=None, y=None) == lm.MOE_LORA_OK
    assert mm(x=None) == EINVAL and mm(y=None) == EINVAL and mm(d=w4(data=None)) == EINVAL
    assert mm(x=at(1, 8)) == EALIGN and mm(y=at(2, 1)) == EALIGN and mm(d=w4(data=at(0, 8))) == EALIGN
    assert mm(y=at(1)) == EINVAL and mm(y=at(0, n - 2)) == EINVAL
    pk = lambda q=at(1), s=at(2), z=None, p=at(3), nb=n, d=d: lib.moe_lora_w4_pack(  # noqa: E731
        ctypes.byref(d), q, s, z, p, nb, None)
    assert pk(q=None) == EINVAL and pk(s=None) == EINVAL and pk(p=None) == EINVAL
    assert pk(z=at(4)) == EINVAL and pk(d=dz, nb=1 << 30) == EINVAL  # zeros exactly with has_zeros
    assert pk(nb=n - 1) == EWS and pk(p=at(3, 4)) == EALIGN and pk(s=at(2, 1)) == EALIGN
    assert pk(p=at(1)) == EINVAL and pk(p=at(2)) == EINVAL


def test_w4_block_arguments(lib):
    g, u, d = w4(64, 32, data=at(0)), w4(64, 32, data=at(1)), w4(32, 64, data=at(2))
    def call(g=g, u=u, d=d, M=2, act=0, x=at(3), ws=at(4), n=1 << 26, y=at(5)):
        return lib.moe_lora_w4_ffn_forward(*(None if t is None else ctypes.byref(t) for t in (g, u, d)), M, act, x,
                                           ws, n, y, None)
    assert call(M=0, x=None, y=None, ws=None) == lm.MOE_LORA_OK
    for over, code in ((dict(g=None), EINVAL), (dict(d=None), EINVAL), (dict(M=-1), EINVAL), (dict(act=2), EINVAL),
                       (dict(M=65537), EUNSUP), (dict(u=w4(56, 32)), EINVAL), (dict(u=w4(64, 40)), EINVAL),
                       (dict(u=w4(64, 32, 64)), EINVAL), (dict(u=w4(64, 32, 32, 1)), EINVAL),
                       (dict(d=w4(40, 64)), EINVAL), (dict(d=w4(32, 72)), EINVAL), (dict(x=None), EINVAL),
                       (dict(y=None), EINVAL), (dict(g=w4(64, 32, data=None)), EINVAL), (dict(ws=None), EWS),
                       (dict(n=2 * 64 * 2 - 1), EWS), (dict(ws=at(4, 8)), EALIGN), (dict(x=at(3, 2)), EALIGN),
                       (dict(y=at(3)), EINVAL), (dict(ws=at(5)), EINVAL), (dict(y=at(2)), EINVAL)):
        assert call(**over) == code, over
    assert lm.moe_lora_w4_ffn_workspace_bytes(-1, 8) == 0 and lm.moe_lora_w4_ffn_workspace_bytes(1, 0) == 0


def test_w4_binding():
    q, s = torch.zeros((16, 32), dtype=torch.uint8), torch.zeros((16, 2), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        lm.moe_lora_w4_pack(q, s, group=32)
    with pytest.raises(ValueError, match="shape"):
        lm.moe_lora_w4_pack(q, s, group=64)
    with pytest.raises(ValueError, match="dtype"):
        lm.moe_lora_w4_pack(q, s.float(), group=32)
    with pytest.raises(ValueError, match="dimensions"):
        lm.moe_lora_w4_pack(q[0], s, group=32)
    with pytest.raises(lm.MoeLoraError):
        lm.moe_lora_w4_pack(q, s, group=48)
    w = lm.W4Weight(16, 64, 32, False)
    with pytest.raises(ValueError, match="shape"):
        lm.moe_lora_w4_matmul(torch.zeros((2, 72), dtype=torch.bfloat16), w, torch.zeros((2, 16)))
    with pytest.raises(ValueError, match="shape"):
        lm.moe_lora_w4_matmul(torch.zeros(64, dtype=torch.bfloat16), w, torch.zeros((2, 16)))


def test_clip_arguments(lib):
    def call(entries=((at(0), at(1), 100, 0),), max_norm=1.0, norm=at(8), ws=at(9), nb=1 << 20, n=None):
        arr = (lm.moe_lora_grad * max(1, len(entries)))(*[lm.moe_lora_grad(*e) for e in entries])
        return lib.moe_lora_clip_grads(arr, len(entries) if n is None else n, max_norm, norm, ws, nb, None)
    assert lib.moe_lora_clip_grads(None, 1, 1.0, at(8), at(9), 1 << 20, None) == EINVAL
    for over, code in (
            (dict(n=-1), EINVAL), (dict(max_norm=-1.0), EINVAL), (dict(max_norm=float("nan")), EINVAL),
            (dict(norm=None), EINVAL), (dict(ws=None), EWS), (dict(nb=64), EWS), (dict(ws=at(9, 4)), EALIGN),
            (dict(norm=at(8, 2)), EALIGN), (dict(entries=[(None, at(1), 5, 0)]), EINVAL),
            (dict(entries=[(at(0), None, 5, 0)]), EINVAL), (dict(entries=[(at(0), at(1), -1, 0)]), EINVAL),
            (dict(entries=[(at(0), at(1), 5, 3)]), EINVAL), (dict(entries=[(at(0, 2), at(1), 5, 0)]), EALIGN),
            (dict(entries=[(at(0), at(1, 1), 5, 1)]), EALIGN),
            (dict(entries=[(at(0), at(1), (1 << 40) + 1, 1)]), EUNSUP),
            # the same tensor twice, in place and not; an output on another's gradient, on its own but shifted,
            # on the norm and on the workspace
            (dict(entries=[(at(0), at(0), 5, 0)] * 2), EINVAL), (dict(entries=[(at(0), at(1), 5, 0)] * 2), EINVAL),
            (dict(entries=[(at(0), at(0), 100, 0), (at(0, 396), at(3), 5, 0)]), EINVAL),
            (dict(entries=[(at(0), at(1), 100, 0), (at(2), at(0, 8), 5, 0)]), EINVAL),
            (dict(entries=[(at(0), at(0, 4), 100, 0)]), EINVAL), (dict(entries=[(at(0), at(8), 100, 0)]), EINVAL),
            (dict(entries=[(at(8), at(1), 1, 0)]), EINVAL), (dict(entries=[(at(0), at(9, 16), 1, 0)]), EINVAL)):
        assert call(**over) == code, over
    assert lm.moe_lora_clip_workspace_bytes(-1) == 0
    assert lm.moe_lora_clip_workspace_bytes(1000) > lm.moe_lora_clip_workspace_bytes(1) > 0


def test_clip_binding():
    with pytest.raises(ValueError, match="out holds"):
        lm.GradSet([torch.zeros(3)], out=[])
    with pytest.raises(ValueError, match="dtype"):
        lm.GradSet([torch.zeros(3, dtype=torch.float64)])
    with pytest.raises(ValueError, match="device tensors"):
        lm.GradSet([torch.zeros(3)])
    with pytest.raises(ValueError, match="dtype"):
        lm.GradSet([torch.zeros(3)], out=[torch.zeros(3, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="contiguous"):
        lm.GradSet([torch.zeros((4, 3)).t()])


def test_tensors_of_another_device(monkeypatch):
    """Operands on a GPU that is not the current one are refused."""
    class Far:
        dtype, shape, is_cuda, device = torch.bfloat16, (2, 16), True, torch.device("cuda", 1)
        def is_contiguous(self):
            return True
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        lm._check_tensors([("x", Far(), (2, 16), "bfloat16")])

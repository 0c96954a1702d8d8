"""The dense operators' host side at the edges of what their contracts allow,
without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import lora_moe_amd as lm

# addresses far apart that nothing ever reads: every call here is refused
BASE, STEP = 1 << 40, 1 << 36


@pytest.mark.parametrize("N,M,K", [(1, 9, 1024), (2, 9, 2048), (3, 10, 896), (1, 32, 1024), (2, 16, 1024),
                                   (5, 32, 1024), (64, 9, 2048)])
def test_slabs_of_a_few_bytes_are_asked_for(N, M, K):
    """A product that cannot do without a workspace never reports the 256
    bytes of one that can."""
    lib = lm.load_library()
    d = lm.moe_lora_w4(BASE, N, K, 128, 0)
    need = lib.moe_lora_w4_workspace_bytes(ctypes.byref(d), M)
    call = lambda ws, n: lib.moe_lora_w4_matmul(ctypes.byref(d), M, BASE + STEP, ws, n, BASE + 2 * STEP,  # noqa: E731
                                                None)
    assert call(None, 0) == lm.MOE_LORA_EWORKSPACE and call(BASE + 3 * STEP, 0) == lm.MOE_LORA_EWORKSPACE
    assert need >= 512


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeTensor:
    """Memory of the stream that was current when it was allocated."""
    dtype, device, is_cuda = torch.uint8, torch.device("cuda", 0), True

    def __init__(self, shape, pool):
        self.shape, self.pool, self.used_on = tuple(shape), pool, set()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def data_ptr(self):
        return id(self)

    def detach(self):
        return self

    def record_stream(self, stream):
        self.used_on.add(stream.cuda_stream)


class Streams:
    """Stands in for the GPU's streams and allocator; made: what the code
    under test allocated; calls: the stream of each library call."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.calls = 3, [], []
        outer = self

        class Scope:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, outer.now = outer.now, self.stream.cuda_stream

            def __exit__(self, *exc):
                outer.now = self.before

        class Library:
            def __getattr__(self, name):
                if name.endswith("_bytes"):
                    return lambda *a: 4096
                return lambda *a: outer.calls.append(a[-1]) or 0

        def empty(shape, *more, **kw):
            t = FakeTensor((shape,) if isinstance(shape, int) else shape, outer.now)
            outer.made.append(t)
            return t

        monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: FakeStream(handle or 99))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
        monkeypatch.setattr(torch.cuda, "stream", Scope)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(outer.now))
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape))
        monkeypatch.setattr(lm, "load_library", lambda *a: Library())
        monkeypatch.setattr(lm, "_check_tensors", lambda specs: None)
        monkeypatch.setattr(lm, "_stream", lambda s: outer.now if s is None else getattr(s, "cuda_stream", s))


@pytest.mark.parametrize("stream", [FakeStream(7), 7, FakeStream(3), 3, None, 0])
def test_buffers_are_memory_of_the_stream_that_writes_them(monkeypatch, stream):
    s = Streams(monkeypatch)
    want = 3 if stream is None else getattr(stream, "cuda_stream", stream)
    t = lambda *shape: FakeTensor(shape, 3)  # noqa: E731
    w = lm.moe_lora_w4_pack(t(64, 32), t(64, 1), group=64, stream=stream)
    y = lm.gated_ffn(t(4, 64), t(64, 64), t(64, 32), stream=stream)
    lm.moe_lora_w4_matmul(t(4, 64), w, t(4, 64), stream=stream)
    assert s.calls == [want] * 3 and len(s.made) == 4
    assert [m.pool for m in s.made] == [want] * 4
    if want != 3:  # what the caller gets is also used on the stream that is current there
        assert w.packed.used_on == {3} and y.used_on == {3}
    assert s.now == 3


def test_a_set_of_gradients_has_a_workspace_for_each_stream(monkeypatch):
    """Listed on one stream and clipped on others, given or current: each
    call writes memory of its own stream, and the same one every time."""
    s = Streams(monkeypatch)
    g = FakeTensor((8,), 3)
    g.dtype = torch.float32
    norm, seen = FakeTensor((1,), 3), []
    library = lm.load_library()
    monkeypatch.setattr(type(library), "moe_lora_clip_grads", lambda self, *a: seen.append((a[4], a[6])) or 0,
                        raising=False)
    gs = lm.GradSet([g])
    for now, given in ((3, None), (3, 7), (9, None), (3, None), (9, 7), (3, 9)):
        s.now = now
        lm.moe_lora_clip_grads(gs, 1.0, norm, stream=given)
    pools = {m.data_ptr(): m.pool for m in s.made}
    assert [pools[ws] for ws, _ in seen] == [stream for _, stream in seen] == [3, 7, 9, 3, 7, 9]
    assert len(s.made) == 3
    s.now = 3
    lm.moe_lora_clip_grads([g], 1.0, norm, stream=11)
    assert s.made[-1].pool == 11 and seen[-1] == (s.made[-1].data_ptr(), 11)


@pytest.mark.parametrize("stream", [FakeStream(7), 7, None])
def test_the_layer_in_one_call_allocates_on_its_stream(monkeypatch, stream):
    s = Streams(monkeypatch)
    monkeypatch.setattr(lm, "check_operands", lambda *a, **kw: None)
    t = lambda *shape: FakeTensor(shape, 3)  # noqa: E731
    streams = []
    monkeypatch.setattr(lm, "moe_lora_align", lambda *a: streams.append(a[-1]))
    monkeypatch.setattr(lm, "moe_lora_forward", lambda *a: streams.append(a[-1]))
    y = lm.fused_moe_lora(t(4, 64), t(4, 2), t(4, 2), t(4), t(8, 64, 64), t(8, 64, 32), t(2, 8, 16, 64),
                          t(2, 8, 64, 16), t(2, 8, 16, 32), t(2, 8, 64, 16), stream=stream)
    want = 3 if stream is None else 7
    assert streams == [stream] * 2 and [m.pool for m in s.made] == [want] * 2 and y is s.made[1]


CSRC = os.path.join(lm.PKG, "csrc")


def test_assembly_names_the_registers_it_sets():
    """A block of assembly that sets m0 says so to the compiler."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for block in re.findall(r"\basm\s*(?:volatile)?\s*\((.*?)\);", text, re.S):
            if re.search(r"\bs_\w+ m0\b", block):
                found += 1
                assert '"m0"' in block.rsplit(":", 1)[1], (name, block)
    assert found


def test_copies_keep_their_distance_from_vector_writes(tmp_path):
    """A vector instruction that writes a scalar register needs five wait
    states before a memory instruction that reads it; the compiler does not
    see into the copies' assembly, so what it puts before them is checked."""
    from lora_moe_amd import build
    out = str(tmp_path / "ffn_gemm.s")
    subprocess.run([build.HIPCC, *build.FLAGS, "-w", "-S", "--cuda-device-only",
                    os.path.join(CSRC, "ffn_gemm.hip"), "-o", out], check=True, capture_output=True)

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
    assert copies > 500

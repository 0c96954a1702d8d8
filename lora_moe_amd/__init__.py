"""Python binding of the MoE-LoRA C ABI (``include/moe_lora.h``).

Argument marshalling only: every step of the layer runs in the HIP kernels of
``libmoe_lora.so``.  Functions carry the C names; tensors are torch tensors on
the current HIP device (PyTorch supplies device memory and streams).  Loading
fails loudly when the library has not been built -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_lora.so")
TUNING_PATH = os.path.join(PKG, "tuning", "gfx950.json")

MOE_LORA_OK = 0
MOE_LORA_EINVAL = -1
MOE_LORA_EALIGN = -2
MOE_LORA_EWORKSPACE = -3
MOE_LORA_EUNSUPPORTED = -4
MOE_LORA_EHIP = -5
MOE_LORA_ACT_SILU = 0
MOE_LORA_ACT_GELU = 1
MOE_LORA_F32 = 0
MOE_LORA_BF16 = 1
MOE_LORA_F16 = 2
MOE_LORA_NOALLOC_WORKSPACE_BYTES = 64 << 20  # the static workspace of moe_lora_forward_noalloc

_lib = None


class MoeLoraError(RuntimeError):
    def __init__(self, func: str, code: int):
        self.code = code
        super().__init__(f"{func} failed: {moe_lora_status_str(code)} ({code})")


KNOBS = ("shrink_splits", "shrink_zblocks", "down_splits", "tile_order", "expand_mode")


class moe_lora_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("L", ctypes.c_int32),
                ("r", ctypes.c_int32), ("block_m", ctypes.c_int32),
                ("lora_scale", ctypes.c_float)] + [(k, ctypes.c_int32) for k in KNOBS]

    def __repr__(self):
        return ("moe_lora_shape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_)
                + ")")


class moe_lora_views(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "sorted_ids", "expert_off", "seg_start", "seg_cnt", "block_expert", "pos_of_pair",
        "num_padded", "err_count", "z_gu", "z_down", "h", "d")] + [
        ("cap_rows", ctypes.c_int64), ("cap_blocks", ctypes.c_int64), ("block_m", ctypes.c_int32),
        ("d_splits", ctypes.c_int32), ("h_lo", ctypes.c_void_p)]


ALIGN_VIEW_FIELDS = ("sorted_ids", "expert_off", "seg_start", "seg_cnt", "block_expert",
                     "pos_of_pair", "num_padded", "err_count")


class moe_lora_align_ptrs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ALIGN_VIEW_FIELDS]


class moe_lora_tune_entry(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows_per_expert", "H", "I", "E", "r", "L", "block_m")
                + KNOBS]


class moe_lora_ffn_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "act")]


class moe_lora_w4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in (
        "N", "K", "group", "has_zeros")]


class moe_lora_grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class moe_lora_sort_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "topk", "dtype")]


class moe_lora_proj_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "K", "N", "L", "r")] + [("lora_scale", ctypes.c_float)]


# An entry's tuned configuration applies to shapes within this distance of
# its key (sum over rows per expert (x4), H, I, E, r, L of |log2 ratio|):
# e.g. a shape with half or twice the entry's rows per expert and the same
# sizes otherwise; farther shapes keep the built-in choice.
TUNE_MAX_DIST = 4.0


def make_shape(T, H, I, E, topk, L, r, block_m=0, lora_scale=1.0, tuning=None,
               max_dist=TUNE_MAX_DIST, **knobs) -> moe_lora_shape:
    """The shape struct (knobs: shrink_splits, shrink_zblocks, down_splits,
    tile_order, expand_mode; 0 = the library's choice).  With a tuning table
    (load_tuning), every field left at 0 is taken from the table's nearest
    entry within max_dist (moe_lora_tune_apply)."""
    s = moe_lora_shape(int(T), int(H), int(I), int(E), int(topk), int(L), int(r), int(block_m),
                       float(lora_scale), *(int(knobs.pop(k, 0)) for k in KNOBS))
    if knobs:
        raise TypeError(f"unknown shape fields {sorted(knobs)}")
    if tuning is not None:
        s = moe_lora_tune_apply(s, tuning, max_dist)
    return s


def load_tuning(path: str = TUNING_PATH):
    """Entries of a tile-configuration table written by ``lora_moe_amd.tune``
    (JSON), as the C array moe_lora_tune_apply reads (knobs missing from an
    entry are 0)."""
    import json
    with open(path) as f:
        doc = json.load(f)
    rows = doc["entries"]
    arr = (moe_lora_tune_entry * max(1, len(rows)))()
    for i, e in enumerate(rows):
        arr[i] = moe_lora_tune_entry(*(int(e.get(n, 0)) for n, _ in moe_lora_tune_entry._fields_))
    return arr, len(rows)


def moe_lora_tune_block_m(shape: moe_lora_shape, tuning, max_dist: float = 0.0) -> int:
    table, n = tuning
    return load_library().moe_lora_tune_block_m(ctypes.byref(shape), table, int(n), float(max_dist))


def moe_lora_tune_apply(shape: moe_lora_shape, tuning, max_dist: float = 0.0) -> moe_lora_shape:
    """A copy of ``shape`` with block_m and the knobs it leaves at 0 taken
    from the nearest table entry."""
    table, n = tuning
    out = moe_lora_shape()
    _check("moe_lora_tune_apply", min(0, load_library().moe_lora_tune_apply(
        ctypes.byref(shape), table, int(n), float(max_dist), ctypes.byref(out))))
    return out


def load_library(path: str = LIB_PATH):
    """Load libmoe_lora.so (raises when it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} not found: build the HIP library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, sp = ctypes.c_void_p, ctypes.POINTER(moe_lora_shape)
    i32 = ctypes.c_int
    lib.moe_lora_resolve_block_m.argtypes = [sp]
    lib.moe_lora_resolve_block_m.restype = i32
    lib.moe_lora_tune_block_m.argtypes = [sp, ctypes.POINTER(moe_lora_tune_entry), ctypes.c_int32,
                                          ctypes.c_float]
    lib.moe_lora_tune_block_m.restype = i32
    lib.moe_lora_tune_apply.argtypes = [sp, ctypes.POINTER(moe_lora_tune_entry), ctypes.c_int32,
                                        ctypes.c_float, sp]
    lib.moe_lora_tune_apply.restype = i32
    lib.moe_lora_workspace_bytes.argtypes = [sp]
    lib.moe_lora_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_lora_align.argtypes = [sp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.moe_lora_align.restype = i32
    lib.moe_lora_align_timed.argtypes = [sp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.moe_lora_align_timed.restype = i32
    lib.moe_lora_align_view.argtypes = [sp, vp, ctypes.POINTER(moe_lora_align_ptrs)]
    lib.moe_lora_align_view.restype = i32
    lib.moe_lora_route.argtypes = [sp, vp, vp, vp, vp]
    lib.moe_lora_route.restype = i32
    lib.moe_lora_route_align.argtypes = [sp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.moe_lora_route_align.restype = i32
    lib.moe_lora_route_align_timed.argtypes = [sp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.moe_lora_route_align_timed.restype = i32
    lib.moe_lora_workspace_view.argtypes = [sp, vp, ctypes.POINTER(moe_lora_views)]
    lib.moe_lora_workspace_view.restype = i32
    lib.moe_lora_forward.argtypes = [sp] + [vp] * 11 + [ctypes.c_size_t, vp, vp]
    lib.moe_lora_forward.restype = i32
    lib.moe_lora_forward_timed.argtypes = [sp] + [vp] * 11 + [ctypes.c_size_t, vp, vp, vp]
    lib.moe_lora_forward_timed.restype = i32
    lib.moe_lora_forward_noalloc.argtypes = [sp] + [vp] * 11 + [vp]
    lib.moe_lora_forward_noalloc.restype = i32
    lib.moe_lora_device_errors.argtypes = [sp, vp, ctypes.POINTER(ctypes.c_int32), vp]
    lib.moe_lora_device_errors.restype = i32
    lib.moe_lora_status_str.argtypes = [i32]
    lib.moe_lora_status_str.restype = ctypes.c_char_p
    lib.moe_lora_stage_count.argtypes = []
    lib.moe_lora_stage_count.restype = i32
    lib.moe_lora_stage_name.argtypes = [i32]
    lib.moe_lora_stage_name.restype = ctypes.c_char_p
    lib.moe_lora_profiler_create.argtypes = [i32, ctypes.c_uint32, ctypes.POINTER(vp)]
    lib.moe_lora_profiler_create.restype = i32
    lib.moe_lora_profiler_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), i32,
                                           ctypes.POINTER(ctypes.c_int)]
    lib.moe_lora_profiler_read.restype = i32
    lib.moe_lora_profiler_destroy.argtypes = [vp]
    lib.moe_lora_profiler_destroy.restype = None
    fp, wp = ctypes.POINTER(moe_lora_ffn_shape), ctypes.POINTER(moe_lora_w4)
    op, pp = ctypes.POINTER(moe_lora_sort_shape), ctypes.POINTER(moe_lora_proj_shape)
    sz, c32 = ctypes.c_size_t, ctypes.c_int32
    for name, restype, argtypes in (
            ("moe_lora_ffn_workspace_bytes", sz, [fp, i32]),
            ("moe_lora_ffn_forward", i32, [fp] + [vp] * 5 + [sz, vp, vp]),
            ("moe_lora_ffn_backward", i32, [fp] + [vp] * 6 + [sz] + [vp] * 4),
            ("moe_lora_w4_bytes", sz, [wp]),
            ("moe_lora_w4_pack", i32, [wp, vp, vp, vp, vp, sz, vp]),
            ("moe_lora_w4_workspace_bytes", sz, [wp, c32]),
            ("moe_lora_w4_matmul", i32, [wp, c32, vp, vp, sz, vp, vp]),
            ("moe_lora_w4_ffn_workspace_bytes", sz, [c32, c32]),
            ("moe_lora_w4_ffn_forward", i32, [wp, wp, wp, c32, c32, vp, vp, sz, vp, vp]),
            ("moe_lora_clip_workspace_bytes", sz, [c32]),
            ("moe_lora_clip_grads", i32,
             [ctypes.POINTER(moe_lora_grad), c32, ctypes.c_float, vp, vp, sz, vp]),
            ("moe_lora_sort_workspace_bytes", sz, [op]),
            ("moe_lora_sort", i32, [op] + [vp] * 3 + [sz] + [vp] * 5),
            ("moe_lora_sort_backward", i32, [op] + [vp] * 4),
            ("moe_lora_unsort", i32, [op] + [vp] * 5),
            ("moe_lora_unsort_backward", i32, [op] + [vp] * 7),
            ("moe_lora_route_backward", i32, [sp] + [vp] * 5),
            ("moe_lora_proj_workspace_bytes", sz, [pp, i32]),
            ("moe_lora_proj_forward", i32, [pp] + [vp] * 8 + [sz, vp, vp]),
            ("moe_lora_proj_backward", i32, [pp] + [vp] * 9 + [sz] + [vp] * 4)):
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, argtypes
    _lib = lib
    return lib


def _check(func: str, code: int):
    if code != MOE_LORA_OK:
        raise MoeLoraError(func, code)


def _ptr(t, name: str):
    """Device address of a contiguous tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.data_ptr()


def layer_operand_specs(shape) -> dict:
    """Expected (shape, dtype name) of every tensor the calls take, from the
    layer sizes in ``shape``."""
    T, H, I, E, k, L, r = shape.T, shape.H, shape.I, shape.E, shape.topk, shape.L, shape.r
    return dict(
        x=((T, H), "bfloat16"), topk_ids=((T, k), "int32"), topk_weights=((T, k), "float32"),
        lora_ids=((T,), "int32"), W_gu=((E, 2 * I, H), "bfloat16"), W_down=((E, H, I), "bfloat16"),
        A_gu=((L, E, r, H), "bfloat16"), B_gu=((L, E, 2 * I, r), "bfloat16"),
        A_down=((L, E, r, I), "bfloat16"), B_down=((L, E, H, r), "bfloat16"),
        y=((T, H), "bfloat16"), logits=((T, E), "float32"))


def check_operands(shape, workspace=None, **tensors) -> None:
    """Raise ValueError unless every given tensor has the dtype and shape the
    kernels assume for ``shape``, is contiguous, and all of them (workspace
    included) are device tensors on one device; the workspace must be a uint8
    tensor of at least moe_lora_workspace_bytes(shape) bytes.  Runs before
    any launch: a wrong dtype (int64 ids from torch.topk, say) or a short
    weight stack would otherwise be read as something else, or past its end."""
    specs = layer_operand_specs(shape)
    devices = set()
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is required")
        want_shape, want_dtype = specs[name]
        got_dtype = str(t.dtype).replace("torch.", "")
        if got_dtype != want_dtype:
            raise ValueError(f"{name}: dtype {got_dtype}, expected {want_dtype}")
        if tuple(t.shape) != want_shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {want_shape}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        devices.add(t.device)
    if workspace is not None:
        if str(workspace.dtype) != "torch.uint8" or workspace.dim() != 1:
            raise ValueError("workspace must be a 1-D uint8 tensor (alloc_workspace)")
        need = moe_lora_workspace_bytes(shape)
        if need == 0:
            raise MoeLoraError("moe_lora_workspace_bytes", MOE_LORA_EINVAL)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes, the shape needs {need}")
        devices.add(workspace.device)
    for d in devices:
        if d.type != "cuda":
            raise ValueError(f"operands must be device tensors (got one on {d})")
    if len(devices) > 1:
        raise ValueError(f"operands on several devices: {sorted(str(d) for d in devices)}")


def _stream(stream):
    if stream is None:
        import torch
        # the handle without the Stream object around it (0.4 us against 2.7
        # a call, a quarter of a small product's)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return getattr(stream, "cuda_stream", stream)


def moe_lora_status_str(code: int) -> str:
    return load_library().moe_lora_status_str(int(code)).decode()


def moe_lora_resolve_block_m(shape: moe_lora_shape) -> int:
    return load_library().moe_lora_resolve_block_m(ctypes.byref(shape))


def moe_lora_workspace_bytes(shape: moe_lora_shape) -> int:
    return int(load_library().moe_lora_workspace_bytes(ctypes.byref(shape)))


def alloc_workspace(shape: moe_lora_shape, device="cuda"):
    import torch
    n = moe_lora_workspace_bytes(shape)
    if n == 0:
        raise MoeLoraError("moe_lora_workspace_bytes", MOE_LORA_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _prof(profiler):
    return None if profiler is None else profiler.handle


def moe_lora_route(shape, logits, topk_ids, topk_weights, stream=None) -> None:
    """Top-k experts and weights of each token from fp32 logits [T, E] into
    topk_ids [T, k] (int32) and topk_weights [T, k] (fp32)."""
    check_operands(shape, logits=logits, topk_ids=topk_ids, topk_weights=topk_weights)
    _check("moe_lora_route", load_library().moe_lora_route(
        ctypes.byref(shape), _ptr(logits, "logits"), _ptr(topk_ids, "topk_ids"),
        _ptr(topk_weights, "topk_weights"), _stream(stream)))


def moe_lora_route_align(shape, logits, lora_ids, topk_ids, topk_weights, workspace,
                         stream=None, profiler=None) -> None:
    """moe_lora_route then moe_lora_align on the routed ids (one kernel for
    small batches)."""
    check_operands(shape, workspace, logits=logits, lora_ids=lora_ids, topk_ids=topk_ids,
                   topk_weights=topk_weights)
    _check("moe_lora_route_align", load_library().moe_lora_route_align_timed(
        ctypes.byref(shape), _ptr(logits, "logits"), _ptr(lora_ids, "lora_ids"),
        _ptr(topk_ids, "topk_ids"), _ptr(topk_weights, "topk_weights"),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream), _prof(profiler)))


def moe_lora_align(shape, topk_ids, lora_ids, workspace, stream=None, profiler=None) -> None:
    check_operands(shape, workspace, topk_ids=topk_ids, lora_ids=lora_ids)
    _check("moe_lora_align", load_library().moe_lora_align_timed(
        ctypes.byref(shape), _ptr(topk_ids, "topk_ids"), _ptr(lora_ids, "lora_ids"),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream), _prof(profiler)))


def moe_lora_forward(shape, x, topk_ids, topk_weights, lora_ids, W_gu, W_down, A_gu, B_gu,
                     A_down, B_down, workspace, y, stream=None, profiler=None) -> None:
    check_operands(shape, workspace, x=x, topk_ids=topk_ids, topk_weights=topk_weights,
                   lora_ids=lora_ids, W_gu=W_gu, W_down=W_down, A_gu=A_gu, B_gu=B_gu,
                   A_down=A_down, B_down=B_down, y=y)
    _check("moe_lora_forward", load_library().moe_lora_forward_timed(
        ctypes.byref(shape), _ptr(x, "x"), _ptr(topk_ids, "topk_ids"),
        _ptr(topk_weights, "topk_weights"), _ptr(lora_ids, "lora_ids"), _ptr(W_gu, "W_gu"),
        _ptr(W_down, "W_down"), _ptr(A_gu, "A_gu"), _ptr(B_gu, "B_gu"), _ptr(A_down, "A_down"),
        _ptr(B_down, "B_down"), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(y, "y"), _stream(stream),
        _prof(profiler)))


def moe_lora_forward_noalloc(shape, x, topk_ids, topk_weights, lora_ids, W_gu, W_down, A_gu, B_gu,
                             A_down, B_down, y, stream=None) -> None:
    """Align + forward with the library's static workspace (for callers that
    cannot allocate); shapes whose workspace exceeds
    MOE_LORA_NOALLOC_WORKSPACE_BYTES raise MoeLoraError (EWORKSPACE)."""
    check_operands(shape, x=x, topk_ids=topk_ids, topk_weights=topk_weights, lora_ids=lora_ids,
                   W_gu=W_gu, W_down=W_down, A_gu=A_gu, B_gu=B_gu, A_down=A_down, B_down=B_down,
                   y=y)
    _check("moe_lora_forward_noalloc", load_library().moe_lora_forward_noalloc(
        ctypes.byref(shape), _ptr(x, "x"), _ptr(topk_ids, "topk_ids"),
        _ptr(topk_weights, "topk_weights"), _ptr(lora_ids, "lora_ids"), _ptr(W_gu, "W_gu"),
        _ptr(W_down, "W_down"), _ptr(A_gu, "A_gu"), _ptr(B_gu, "B_gu"), _ptr(A_down, "A_down"),
        _ptr(B_down, "B_down"), _ptr(y, "y"), _stream(stream)))


def moe_lora_align_view(shape, workspace) -> dict:
    """Device addresses (ints) of the align outputs in ``workspace``."""
    v = moe_lora_align_ptrs()
    _check("moe_lora_align_view", load_library().moe_lora_align_view(
        ctypes.byref(shape), ctypes.c_void_p(workspace if isinstance(workspace, int)
                                             else workspace.data_ptr()), ctypes.byref(v)))
    return {n: getattr(v, n) for n in ALIGN_VIEW_FIELDS}


def moe_lora_workspace_view(shape, workspace) -> moe_lora_views:
    v = moe_lora_views()
    _check("moe_lora_workspace_view", load_library().moe_lora_workspace_view(
        ctypes.byref(shape), _ptr(workspace, "workspace"), ctypes.byref(v)))
    return v


def workspace_tensors(shape, workspace) -> dict:
    """The workspace regions of ``moe_lora_workspace_view`` as torch views of
    ``workspace`` (a uint8 device tensor)."""
    import torch
    v = moe_lora_workspace_view(shape, workspace)
    base = workspace.data_ptr()
    P = shape.T * shape.topk
    NB = shape.E * (shape.L + 1)
    cap, capb = v.cap_rows, v.cap_blocks

    def region(addr, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        off = addr - base
        return workspace[off:off + nbytes].view(dtype)

    return dict(
        sorted_ids=region(v.sorted_ids, cap, torch.int32),
        expert_off=region(v.expert_off, shape.E + 1, torch.int32),
        seg_start=region(v.seg_start, NB, torch.int32),
        seg_cnt=region(v.seg_cnt, NB, torch.int32),
        block_expert=region(v.block_expert, capb, torch.int32),
        pos_of_pair=region(v.pos_of_pair, P, torch.int32),
        num_padded=region(v.num_padded, 1, torch.int32),
        err_count=region(v.err_count, 1, torch.int32),
        z_gu=region(v.z_gu, cap * shape.r, torch.float32).view(cap, shape.r),
        z_down=region(v.z_down, cap * shape.r, torch.float32).view(cap, shape.r),
        h=region(v.h, cap * shape.I, torch.bfloat16).view(cap, shape.I),
        d=region(v.d, v.d_splits * cap * shape.H, torch.float32).view(v.d_splits, cap, shape.H),
        h_lo=(region(v.h_lo, cap * shape.I, torch.bfloat16).view(cap, shape.I) if v.h_lo else None),
        cap_rows=cap, cap_blocks=capb, block_m=v.block_m, d_splits=v.d_splits)


def moe_lora_device_errors(shape, workspace, stream=None) -> int:
    n = ctypes.c_int32(0)
    _check("moe_lora_device_errors", load_library().moe_lora_device_errors(
        ctypes.byref(shape), _ptr(workspace, "workspace"), ctypes.byref(n), _stream(stream)))
    return int(n.value)


def moe_lora_stage_count() -> int:
    return load_library().moe_lora_stage_count()


def moe_lora_stage_name(i: int) -> str:
    return load_library().moe_lora_stage_name(int(i)).decode()


class Profiler:
    """A caller-owned stage-timing recorder (moe_lora_profiler_create): pass
    it as ``profiler=`` to align / route_align / forward; ``read()`` waits
    for the recorded events and returns the summed milliseconds per stage
    name and the number of recorded calls."""

    def __init__(self, max_calls: int, stages=None):
        mask = 0xFFFFFFFF
        if stages is not None:
            names = [moe_lora_stage_name(i) for i in range(moe_lora_stage_count())]
            mask = 0
            for st in stages:
                mask |= 1 << names.index(st)
        h = ctypes.c_void_p()
        _check("moe_lora_profiler_create", load_library().moe_lora_profiler_create(
            int(max_calls), mask, ctypes.byref(h)))
        self.handle = h

    def read(self) -> tuple[dict, int]:
        n = moe_lora_stage_count()
        arr = (ctypes.c_float * n)()
        calls = ctypes.c_int(0)
        _check("moe_lora_profiler_read", load_library().moe_lora_profiler_read(
            self.handle, arr, n, ctypes.byref(calls)))
        return {moe_lora_stage_name(i): float(arr[i]) for i in range(n)}, int(calls.value)

    def close(self) -> None:
        if self.handle:
            load_library().moe_lora_profiler_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fused_moe_lora(x, topk_ids, topk_weights, lora_ids, W_gu, W_down, A_gu, B_gu, A_down, B_down,
                   lora_scale=1.0, block_m=0, workspace=None, y=None, stream=None):
    """Align + forward on the current stream; returns y [T, H] (bf16).

    x [T,H] bf16; topk_ids [T,k] int32; topk_weights [T,k] fp32; lora_ids [T]
    int32; W_gu [E,2I,H]; W_down [E,H,I]; A_gu [L,E,r,H]; B_gu [L,E,2I,r];
    A_down [L,E,r,I]; B_down [L,E,H,r] (all bf16)."""
    import torch
    for name, t, nd in (("x", x, 2), ("topk_ids", topk_ids, 2), ("W_gu", W_gu, 3), ("A_gu", A_gu, 4)):
        if t.dim() != nd:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected {nd}")
    T, H = x.shape
    E, twoI, _ = W_gu.shape
    L, _, r, _ = A_gu.shape
    shape = make_shape(T, H, twoI // 2, E, topk_ids.shape[1], L, r, block_m, lora_scale)
    check_operands(shape, x=x, topk_ids=topk_ids, topk_weights=topk_weights, lora_ids=lora_ids,
                   W_gu=W_gu, W_down=W_down, A_gu=A_gu, B_gu=B_gu, A_down=A_down, B_down=B_down)
    if workspace is None:
        workspace = _allocated_on(stream, lambda: alloc_workspace(shape, x.device))
    if y is None:
        y = _allocated_on(stream, lambda: torch.empty((T, H), dtype=torch.bfloat16, device=x.device),
                          returned=True)
    moe_lora_align(shape, topk_ids, lora_ids, workspace, stream)
    moe_lora_forward(shape, x, topk_ids, topk_weights, lora_ids, W_gu, W_down, A_gu, B_gu, A_down,
                     B_down, workspace, y, stream)
    return y


# ------------------------------------------------------------------ dense blocks

_ACTS = {"silu": MOE_LORA_ACT_SILU, "gelu": MOE_LORA_ACT_GELU}
_GRAD_TYPES = {"torch.float32": MOE_LORA_F32, "torch.bfloat16": MOE_LORA_BF16,
               "torch.float16": MOE_LORA_F16}


def _act_code(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"act: {act!r}, expected one of {sorted(_ACTS)}")
    return _ACTS[act]


def _check_tensors(specs) -> None:
    """Raise ValueError unless each (name, tensor, shape, dtype) matches, is
    contiguous, and all tensors lie on the current HIP device.  A shape of
    None is not compared."""
    import torch
    for name, t, shape, dtype in specs:
        if t is None:
            raise ValueError(f"{name} is required")
        if t.dtype is not getattr(torch, dtype):
            raise ValueError(f"{name}: dtype {str(t.dtype)[6:]}, expected {dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for name, t, _, _ in specs:
        if not t.is_cuda:
            raise ValueError(f"operands must be device tensors ({name} is on {t.device})")
    dev = torch.cuda.current_device() if specs else None
    for name, t, _, _ in specs:
        if t.device.index != dev:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _address(name, t):
    """Device address of an operand that may be left out (None).  One without
    memory (a fake tensor, torch's zeros that are none) has the address 0 and
    would pass for left out."""
    if t is None:
        return None
    p = t.data_ptr()
    if not p and t.numel():
        raise ValueError(f"{name} has no memory")
    return p


def _allocated_on(stream, make, returned=False):
    """What make() allocates, as memory of ``stream``: the allocator hands a
    block of one stream to the next user in that stream's order alone, so
    memory that work on ``stream`` writes has to come from its own pool, both
    when it is taken (earlier users may still run) and when it is let go.
    returned: the caller uses it on the current stream afterwards."""
    if stream is None or _stream(stream) == _stream(None):
        return make()
    import torch
    handle = _stream(stream)
    if not isinstance(stream, torch.cuda.Stream):
        # (an ExternalStream of address 0 is not the default stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = make()
    if returned:
        t.record_stream(torch.cuda.current_stream())
    return t


def _check_workspace(workspace, need: int, what: str):
    if workspace is None:
        raise ValueError(f"workspace is required ({what})")
    if str(workspace.dtype) != "torch.uint8" or workspace.dim() != 1:
        raise ValueError(f"workspace must be a 1-D uint8 tensor ({what})")
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
    return ("workspace", workspace, None, "uint8")


def make_ffn_shape(T, H, I, act="silu") -> moe_lora_ffn_shape:
    """Sizes of a gated feed-forward block; act: "silu" or "gelu" (tanh form)."""
    return moe_lora_ffn_shape(int(T), int(H), int(I), _act_code(act))


def moe_lora_ffn_workspace_bytes(shape: moe_lora_ffn_shape, backward: bool = True) -> int:
    return int(load_library().moe_lora_ffn_workspace_bytes(ctypes.byref(shape), int(bool(backward))))


def alloc_ffn_workspace(shape: moe_lora_ffn_shape, backward: bool = True, device="cuda"):
    """Workspace of moe_lora_ffn_forward and (backward) moe_lora_ffn_backward."""
    import torch
    n = moe_lora_ffn_workspace_bytes(shape, backward)
    if n == 0:
        raise MoeLoraError("moe_lora_ffn_workspace_bytes", MOE_LORA_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_lora_ffn_forward(shape, x, W_gu, W_down, workspace, y, gu=None, stream=None) -> None:
    """y = (act(x Wg^T) * (x Wu^T)) W_down^T; with gu ([T, 2I] fp32) the
    pre-activations are kept there for moe_lora_ffn_backward."""
    T, H, I = shape.T, shape.H, shape.I
    specs = [("x", x, (T, H), "bfloat16"), ("W_gu", W_gu, (2 * I, H), "bfloat16"),
             ("W_down", W_down, (H, I), "bfloat16"), ("y", y, (T, H), "bfloat16"),
             _check_workspace(workspace, moe_lora_ffn_workspace_bytes(shape, False),
                              "alloc_ffn_workspace")]
    if gu is not None:
        specs.append(("gu", gu, (T, 2 * I), "float32"))
    _check_tensors(specs)
    _check("moe_lora_ffn_forward", load_library().moe_lora_ffn_forward(
        ctypes.byref(shape), x.data_ptr(), W_gu.data_ptr(), W_down.data_ptr(),
        _address("gu", gu), workspace.data_ptr(), workspace.numel(),
        y.data_ptr(), _stream(stream)))


def moe_lora_ffn_backward(shape, dy, x, gu, W_gu, W_down, workspace, dx=None, dW_gu=None,
                          dW_down=None, stream=None) -> None:
    """Gradients of the block from dy and the kept gu into those of dx, dW_gu
    and dW_down that are given (overwritten)."""
    T, H, I = shape.T, shape.H, shape.I
    specs = [("dy", dy, (T, H), "bfloat16"), ("x", x, (T, H), "bfloat16"),
             ("gu", gu, (T, 2 * I), "float32"), ("W_gu", W_gu, (2 * I, H), "bfloat16"),
             ("W_down", W_down, (H, I), "bfloat16"),
             _check_workspace(workspace, moe_lora_ffn_workspace_bytes(shape, True),
                              "alloc_ffn_workspace")]
    outs = (("dx", dx, (T, H)), ("dW_gu", dW_gu, (2 * I, H)), ("dW_down", dW_down, (H, I)))
    specs += [(n, t, s, "bfloat16") for n, t, s in outs if t is not None]
    _check_tensors(specs)
    _check("moe_lora_ffn_backward", load_library().moe_lora_ffn_backward(
        ctypes.byref(shape), dy.data_ptr(), x.data_ptr(), gu.data_ptr(), W_gu.data_ptr(),
        W_down.data_ptr(), workspace.data_ptr(), workspace.numel(),
        *[_address(n, t) for n, t, _ in outs], _stream(stream)))


def gated_ffn(x, W_gu, W_down, act="silu", workspace=None, y=None, stream=None):
    """The block's forward on the current stream (or ``stream``); returns y
    [T, H] (bf16).  x [T,H], W_gu [2I,H], W_down [H,I], all bf16.  Like every
    call here it records nothing for autograd, whatever its operands require:
    a training program calls moe_lora_ffn_forward with gu and
    moe_lora_ffn_backward itself."""
    import torch
    for name, t in (("x", x), ("W_gu", W_gu)):
        if t.dim() != 2:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected 2")
    shape = make_ffn_shape(x.shape[0], x.shape[1], W_gu.shape[0] // 2, act)
    if workspace is None:
        workspace = _allocated_on(stream, lambda: alloc_ffn_workspace(shape, False, x.device))
    if y is None:
        y = _allocated_on(stream, lambda: torch.empty_like(x), returned=True)
    moe_lora_ffn_forward(shape, x, W_gu, W_down, workspace, y, stream=stream)
    return y


class W4Weight:
    """A packed 4-bit matrix [N, K] (moe_lora_w4_pack): its sizes and its
    device buffer."""

    def __init__(self, N, K, group, has_zeros):
        self.desc = moe_lora_w4(None, int(N), int(K), int(group), int(has_zeros))
        self.packed = None

    N = property(lambda self: self.desc.N)
    K = property(lambda self: self.desc.K)
    group = property(lambda self: self.desc.group)
    has_zeros = property(lambda self: bool(self.desc.has_zeros))

    def _spec(self, name):
        return (name, self.packed, None, "uint8")


def moe_lora_w4_bytes(w: W4Weight) -> int:
    return int(load_library().moe_lora_w4_bytes(ctypes.byref(w.desc)))


def moe_lora_w4_pack(q, scales, zeros=None, group=128, stream=None) -> W4Weight:
    """Lays out 4-bit weights q [N, K/2] uint8 (even k in the low half) with
    scales [N, ceil(K/group)] bf16 and zero points [N, ceil(K/group)] uint8
    (0..15; None: 8 everywhere) for moe_lora_w4_matmul; done once per matrix."""
    import torch
    if q.dim() != 2:
        raise ValueError(f"q: {q.dim()} dimensions, expected 2")
    N, K = q.shape[0], 2 * q.shape[1]
    w = W4Weight(N, K, group, zeros is not None)
    n = moe_lora_w4_bytes(w)
    if n == 0:
        raise MoeLoraError("moe_lora_w4_bytes", MOE_LORA_EALIGN if K % 8 else MOE_LORA_EINVAL)
    G = (K + group - 1) // group
    specs = [("q", q, (N, K // 2), "uint8"), ("scales", scales, (N, G), "bfloat16")]
    if zeros is not None:
        specs.append(("zeros", zeros, (N, G), "uint8"))
    _check_tensors(specs)
    w.packed = _allocated_on(stream, lambda: torch.empty(n, dtype=torch.uint8, device=q.device),
                             returned=True)
    w.desc.data = w.packed.data_ptr()
    _check("moe_lora_w4_pack", load_library().moe_lora_w4_pack(
        ctypes.byref(w.desc), q.data_ptr(), scales.data_ptr(),
        _address("zeros", zeros), w.packed.data_ptr(), n, _stream(stream)))
    return w


def moe_lora_w4_workspace_bytes(w: W4Weight, M: int) -> int:
    return int(load_library().moe_lora_w4_workspace_bytes(ctypes.byref(w.desc), int(M)))


def moe_lora_w4_matmul(x, w: W4Weight, y, workspace=None, stream=None) -> None:
    """y [M, N] = x [M, K] w^T (bf16 rows, packed 4-bit weights).  workspace:
    moe_lora_w4_workspace_bytes(w, M) bytes (uint8); None: allocated here."""
    import torch
    M = x.shape[0] if x.dim() == 2 else -1
    specs = [("x", x, (M, w.K), "bfloat16"), ("y", y, (M, w.N), "bfloat16"), w._spec("w")]
    need = moe_lora_w4_workspace_bytes(w, M)
    if workspace is not None:
        specs.append(_check_workspace(workspace, need, "moe_lora_w4_workspace_bytes"))
    _check_tensors(specs)
    if workspace is None and need > 256:  # 256: none is used
        workspace = _allocated_on(
            stream, lambda: torch.empty(need, dtype=torch.uint8, device=x.device))
    _check("moe_lora_w4_matmul", load_library().moe_lora_w4_matmul(
        ctypes.byref(w.desc), M, x.data_ptr(), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), y.data_ptr(), _stream(stream)))


def moe_lora_w4_ffn_workspace_bytes(M, I) -> int:
    return int(load_library().moe_lora_w4_ffn_workspace_bytes(int(M), int(I)))


def alloc_w4_ffn_workspace(M, I, device="cuda"):
    import torch
    n = moe_lora_w4_ffn_workspace_bytes(M, I)
    if n == 0:
        raise MoeLoraError("moe_lora_w4_ffn_workspace_bytes", MOE_LORA_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_lora_w4_ffn_forward(x, gate: W4Weight, up: W4Weight, down: W4Weight, workspace, y,
                            act="silu", stream=None) -> None:
    """y = (act(x gate^T) * (x up^T)) down^T on packed 4-bit weights."""
    M = x.shape[0] if x.dim() == 2 else -1
    _check_tensors([("x", x, (M, gate.K), "bfloat16"), ("y", y, (M, down.N), "bfloat16"),
                    gate._spec("gate"), up._spec("up"), down._spec("down"),
                    _check_workspace(workspace, moe_lora_w4_ffn_workspace_bytes(M, gate.N),
                                     "alloc_w4_ffn_workspace")])
    _check("moe_lora_w4_ffn_forward", load_library().moe_lora_w4_ffn_forward(
        ctypes.byref(gate.desc), ctypes.byref(up.desc), ctypes.byref(down.desc), M, _act_code(act),
        x.data_ptr(), workspace.data_ptr(), workspace.numel(), y.data_ptr(), _stream(stream)))


class GradSet:
    """The gradients of one training program for moe_lora_clip_grads: checked
    and listed once, kept as long as the program uses these tensors (a tensor
    that is given other memory, by ``.data = ``, needs a new set).  out: where
    the clipped gradients go (like ``grads``); None: in place.  A set has one
    workspace for each stream that it is used on, kept as long as the set: its
    calls on one stream follow one another, as do the replays of the graphs
    that it was captured into on one stream."""

    def __init__(self, grads, out=None):
        import torch
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"out holds {len(self.out)} tensors, grads {len(self.grads)}")
        n = len(self.grads)
        self._arr = (moe_lora_grad * max(1, n))()
        specs = []
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            if str(g.dtype) not in _GRAD_TYPES:
                raise ValueError(f"grads[{i}]: dtype {str(g.dtype)[6:]}, expected float32, bfloat16 or "
                                 "float16")
            dtype, shape = str(g.dtype)[6:], tuple(g.shape)
            specs += [(f"grads[{i}]", g, shape, dtype), (f"out[{i}]", o, shape, dtype)]
            self._arr[i] = moe_lora_grad(g.data_ptr(), o.data_ptr(), g.numel(), _GRAD_TYPES[str(g.dtype)])
        _check_tensors(specs)
        # the listed memory stays allocated, whatever the tensors become
        self._held = [t.detach() for t in self.grads + self.out]
        self._workspaces = {}  # by the stream's handle

    def __len__(self):
        return len(self.grads)

    def _workspace(self, stream):
        handle = _stream(stream)
        if handle not in self._workspaces:
            import torch
            need = moe_lora_clip_workspace_bytes(len(self.grads))
            device = self.grads[0].device if self.grads else "cuda"
            self._workspaces[handle] = _allocated_on(
                stream, lambda: torch.empty(need, dtype=torch.uint8, device=device))
        return self._workspaces[handle]


def moe_lora_clip_workspace_bytes(n: int) -> int:
    return int(load_library().moe_lora_clip_workspace_bytes(int(n)))


def moe_lora_clip_grads(grads, max_norm: float, norm, stream=None) -> None:
    """Scales the gradients (a GradSet, or a list of tensors, in place) by
    min(1, max_norm / (norm + 1e-6)) and writes their global norm to ``norm``
    ([1] fp32, device).  max_norm = inf: the norm only (with out: a copy)."""
    if not isinstance(grads, GradSet):
        grads = GradSet(grads)
    workspace = grads._workspace(stream)
    _check_tensors([("norm", norm, (1,), "float32"), ("workspace", workspace, None, "uint8")])
    _check("moe_lora_clip_grads", load_library().moe_lora_clip_grads(
        grads._arr, len(grads), float(max_norm), norm.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream(stream)))


# ------------------------------------------------------------------ tokens to their experts and back

_ROW_TYPES = {MOE_LORA_F32: "float32", MOE_LORA_BF16: "bfloat16", MOE_LORA_F16: "float16"}
_functions = {}  # the library's: address, type of the shape, kind
_native = None   # the _operands module


def _run(func, shape, args, stream, workspace=None) -> None:
    """Calls the library's ``func`` on the shape, args and the stream; raises
    what is wrong.  args: None, or (name, tensor, sizes, type) for a tensor that
    has to match, be contiguous and lie on the current HIP device; the
    workspace has sizes None and a None behind it for its bytes.  workspace:
    (the bytes needed, as a function; what allocates it)."""
    global _native
    if _native is None:
        import torch
        try:
            from . import _operands
        except ImportError as e:
            raise RuntimeError(f"lora_moe_amd._operands: {e}; build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')") from e
        _native = (_operands.call, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream, _operands.kinds)
    call, device, raw_stream, kinds = _native
    f = _functions.get(func)
    if f is None:
        c = getattr(load_library(), func)
        f = _functions[func] = (ctypes.cast(c, ctypes.c_void_p).value, c.argtypes[0]._type_, kinds[func])
    if not isinstance(shape, f[1]):  # (others have fields of the same names)
        raise TypeError(f"shape: {type(shape).__name__}, expected {f[1].__name__}")
    first = args[0][1]
    code = None
    if first is not None and first.is_cuda:
        dev = device()
        handle = raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)
        code = call(f[0], shape, (*args, handle), dev, f[2])
    if code is None:
        specs = [a for a in args if a is not None and a[2] is not None]
        for a in args:
            if a is not None and a[2] is None:
                specs.append(_check_workspace(a[1], workspace[0](), workspace[1]))
        _check_tensors(specs)
        # as it should be after all (a tensor that DLPack does not take)
        ptrs = [None if a is None else _address(a[0], a[1]) for a in args]
        for i, a in enumerate(args):
            if a is not None and a[2] is None:
                ptrs[i + 1] = a[1].numel()
        code = getattr(load_library(), func)(ctypes.byref(shape), *ptrs, _stream(stream))
    if code != MOE_LORA_OK:
        if code == MOE_LORA_EWORKSPACE:
            _check_workspace(next(a[1] for a in args if a is not None and a[2] is None), workspace[0](), workspace[1])
        _check(func, code)


def _or_none(name, tensor, sizes, dtype):
    return None if tensor is None else (name, tensor, sizes, dtype)


def make_sort_shape(T, H, E, topk, dtype="bfloat16") -> moe_lora_sort_shape:
    """Sizes of a sort by expert; dtype: of the rows, bfloat16, float16 or
    float32 (a torch dtype or its name)."""
    name = str(dtype).replace("torch.", "")
    code = {n: c for c, n in _ROW_TYPES.items()}.get(name)
    if code is None:
        raise ValueError(f"dtype: {name}, expected one of {sorted(_ROW_TYPES.values())}")
    return moe_lora_sort_shape(int(T), int(H), int(E), int(topk), code)


def moe_lora_sort_workspace_bytes(shape: moe_lora_sort_shape) -> int:
    return int(load_library().moe_lora_sort_workspace_bytes(ctypes.byref(shape)))


def alloc_sort_workspace(shape: moe_lora_sort_shape, device="cuda"):
    """Workspace of moe_lora_sort."""
    import torch
    n = moe_lora_sort_workspace_bytes(shape)
    if n == 0:
        raise MoeLoraError("moe_lora_sort_workspace_bytes", MOE_LORA_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _row_type(shape) -> str:
    name = _ROW_TYPES.get(shape.dtype)
    if name is None:
        raise ValueError(f"shape: dtype {shape.dtype}, expected one of {sorted(_ROW_TYPES)}")
    return name


def moe_lora_sort(shape, topk_ids, x, workspace, rows, expert_off, row_of_pair, pair_of_row=None,
                  stream=None) -> None:
    """Sorts the (token, slot) pairs of topk_ids [T, k] by expert and copies
    each pair's token row: rows [T k, H] from x [T, H] (both None: the order
    alone).  expert_off [E+1], row_of_pair [T, k] and pair_of_row [T k] are
    int32 and written."""
    T, k, dtype = shape.T, shape.topk, _row_type(shape)
    both = x is not None or rows is not None
    _run("moe_lora_sort", shape, (
        ("topk_ids", topk_ids, (T, k), "int32"), ("x", x, (T, shape.H), dtype) if both else None,
        ("workspace", workspace, None, "uint8"), None, ("rows", rows, (T * k, shape.H), dtype) if both else None,
        ("expert_off", expert_off, (shape.E + 1,), "int32"), ("row_of_pair", row_of_pair, (T, k), "int32"),
        _or_none("pair_of_row", pair_of_row, (T * k,), "int32")), stream,
        (lambda: moe_lora_sort_workspace_bytes(shape), "alloc_sort_workspace"))


def moe_lora_sort_backward(shape, drows, row_of_pair, dx, stream=None) -> None:
    """dx [T, H]: each token's sum of its pairs' rows of drows [T k, H]."""
    T, H, k, dtype = shape.T, shape.H, shape.topk, _row_type(shape)
    _run("moe_lora_sort_backward", shape, (
        ("drows", drows, (T * k, H), dtype), ("row_of_pair", row_of_pair, (T, k), "int32"),
        ("dx", dx, (T, H), dtype)), stream)


def moe_lora_unsort(shape, rows, row_of_pair, y, weights=None, stream=None) -> None:
    """y [T, H]: each token's sum of its pairs' rows [T k, H], times weights
    [T, k] (fp32; None: ones)."""
    T, H, k, dtype = shape.T, shape.H, shape.topk, _row_type(shape)
    _run("moe_lora_unsort", shape, (
        ("rows", rows, (T * k, H), dtype), ("row_of_pair", row_of_pair, (T, k), "int32"),
        _or_none("weights", weights, (T, k), "float32"), ("y", y, (T, H), dtype)), stream)


def moe_lora_unsort_backward(shape, dy, rows, row_of_pair, drows=None, weights=None, dweights=None,
                             stream=None) -> None:
    """Gradients of moe_lora_unsort from dy [T, H] into those of drows [T k,
    H] and dweights [T, k] (fp32) that are given; rows (as given to the
    forward) are needed for dweights alone."""
    T, H, k, dtype = shape.T, shape.H, shape.topk, _row_type(shape)
    _run("moe_lora_unsort_backward", shape, (
        ("dy", dy, (T, H), dtype), _or_none("rows", rows, (T * k, H), dtype),
        ("row_of_pair", row_of_pair, (T, k), "int32"), _or_none("weights", weights, (T, k), "float32"),
        _or_none("drows", drows, (T * k, H), dtype), _or_none("dweights", dweights, (T, k), "float32")), stream)


def moe_lora_route_backward(shape, topk_ids, topk_weights, dweights, dlogits, stream=None) -> None:
    """The gradient of moe_lora_route's weights: dlogits [T, E] from dweights
    [T, k] (both fp32) and what the router wrote."""
    T, k = shape.T, shape.topk
    _run("moe_lora_route_backward", shape, (
        ("topk_ids", topk_ids, (T, k), "int32"), ("topk_weights", topk_weights, (T, k), "float32"),
        ("dweights", dweights, (T, k), "float32"), ("dlogits", dlogits, (T, shape.E), "float32")), stream)


# ------------------------------------------------------------------ a shared projection with adapters


def make_proj_shape(T, K, N, L, r, lora_scale=1.0) -> moe_lora_proj_shape:
    """Sizes of a projection [N, K] that all tokens share, with L adapters of
    rank r beside it."""
    return moe_lora_proj_shape(int(T), int(K), int(N), int(L), int(r), float(lora_scale))


def moe_lora_proj_workspace_bytes(shape: moe_lora_proj_shape, backward: bool = True) -> int:
    return int(load_library().moe_lora_proj_workspace_bytes(ctypes.byref(shape), int(bool(backward))))


def alloc_proj_workspace(shape: moe_lora_proj_shape, backward: bool = True, device="cuda"):
    """Workspace of moe_lora_proj_forward and (backward) moe_lora_proj_backward."""
    import torch
    n = moe_lora_proj_workspace_bytes(shape, backward)
    if n == 0:
        raise MoeLoraError("moe_lora_proj_workspace_bytes", MOE_LORA_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_lora_proj_forward(shape, x, lora_ids, W, A, B, workspace, y, z=None, scales=None, stream=None) -> None:
    """y [T, N] = x W^T + s_l (x A_l^T) B_l^T with each token's own adapter l =
    lora_ids[t] (-1: none), s_l = lora_scale * scales[l]; with z ([T, r] fp32)
    x A_l^T is kept there for moe_lora_proj_backward."""
    T, K, N, L, r = shape.T, shape.K, shape.N, shape.L, shape.r
    _run("moe_lora_proj_forward", shape, (
        ("x", x, (T, K), "bfloat16"), ("lora_ids", lora_ids, (T,), "int32"), ("W", W, (N, K), "bfloat16"),
        ("A", A, (L, r, K), "bfloat16"), ("B", B, (L, N, r), "bfloat16"), _or_none("scales", scales, (L,), "float32"),
        _or_none("z", z, (T, r), "float32"), ("workspace", workspace, None, "uint8"), None,
        ("y", y, (T, N), "bfloat16")), stream,
        (lambda: moe_lora_proj_workspace_bytes(shape, False), "alloc_proj_workspace"))


def moe_lora_proj_backward(shape, dy, x, lora_ids, z, W, A, B, workspace, dx=None, dA=None, dB=None, scales=None,
                           stream=None) -> None:
    """Gradients of the projection from dy and the kept z into those of dx, dA
    and dB that are given (overwritten); W is frozen."""
    T, K, N, L, r = shape.T, shape.K, shape.N, shape.L, shape.r
    _run("moe_lora_proj_backward", shape, (
        ("dy", dy, (T, N), "bfloat16"), ("x", x, (T, K), "bfloat16"), ("lora_ids", lora_ids, (T,), "int32"),
        ("z", z, (T, r), "float32"), ("W", W, (N, K), "bfloat16"), ("A", A, (L, r, K), "bfloat16"),
        ("B", B, (L, N, r), "bfloat16"), _or_none("scales", scales, (L,), "float32"),
        ("workspace", workspace, None, "uint8"), None, _or_none("dx", dx, (T, K), "bfloat16"),
        _or_none("dA", dA, (L, r, K), "bfloat16"), _or_none("dB", dB, (L, N, r), "bfloat16")), stream,
        (lambda: moe_lora_proj_workspace_bytes(shape, True), "alloc_proj_workspace"))


def lora_projection(x, lora_ids, W, A, B, lora_scale=1.0, scales=None, workspace=None, y=None, stream=None):
    """The projection's forward on the current stream (or ``stream``); returns
    y [T, N] (bf16).  x [T,K], W [N,K], A [L,r,K], B [L,N,r], all bf16;
    lora_ids [T] int32; scales [L] fp32 or None.  It records nothing for
    autograd (see gated_ffn)."""
    import torch
    for name, t, nd in (("x", x, 2), ("W", W, 2), ("A", A, 3)):
        if t.dim() != nd:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected {nd}")
    shape = make_proj_shape(x.shape[0], x.shape[1], W.shape[0], A.shape[0], A.shape[1], lora_scale)
    if workspace is None:
        workspace = _allocated_on(stream, lambda: alloc_proj_workspace(shape, False, x.device))
    if y is None:
        y = _allocated_on(stream, lambda: torch.empty((shape.T, shape.N), dtype=torch.bfloat16, device=x.device),
                          returned=True)
    moe_lora_proj_forward(shape, x, lora_ids, W, A, B, workspace, y, scales=scales, stream=stream)
    return y


__all__ = [n for n in dir() if n.startswith("moe_lora") or n in (
    "make_shape", "alloc_workspace", "workspace_tensors", "fused_moe_lora", "load_library",
    "make_ffn_shape", "alloc_ffn_workspace", "gated_ffn",
    "W4Weight", "alloc_w4_ffn_workspace", "GradSet", "make_sort_shape", "alloc_sort_workspace",
    "make_proj_shape", "alloc_proj_workspace", "lora_projection",
    "MoeLoraError", "Profiler", "check_operands", "layer_operand_specs")]

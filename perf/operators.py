"""The operators beside the MoE-LoRA layer, as cases that can be timed and compared:

  ffn     the gated feed-forward block, forward only (prefill and decode)
  train   the same block forward and backward: y, dx and both weight gradients
  w4      a product of a few rows with 4-bit weights and group scales
  w4ffn   the gated block on 4-bit weights, for the tokens of a decode batch
  clip    the global norm of many gradient tensors, and the clipped gradients

``run`` computes them in plain torch operations in 32 bits, or, with ``own``
set, through the library's entry points.
"""
import math

import torch

own = False

GELU_C = math.sqrt(2.0 / math.pi)
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one request through a dense block: the weight stream
        dict(name="ffn_one_token", op="ffn", T=1, H=4096, I=11008, act="silu"),
        # a decode batch through a wide dense block
        dict(name="ffn_decode_32", op="ffn", T=32, H=5120, I=25600, act="silu"),
        # a prefill of several requests; the token count is nobody's multiple
        dict(name="ffn_prefill", op="ffn", T=2047, H=5120, I=25600, act="silu"),
        # a block of a test model: what launches and latency cost
        dict(name="train_tiny", op="train", T=64, H=256, I=512, act="silu"),
        # a small model's micro-batch with ragged sizes, gelu gating
        dict(name="train_ragged", op="train", T=1001, H=2880, I=2880, act="gelu"),
        # a full training micro-batch
        dict(name="train_large", op="train", T=8192, H=4096, I=11008, act="silu"),
        # one token against a projection: the smallest product
        dict(name="w4_one_row", op="w4", M=1, N=4096, K=4096, group=128, zeros=False),
        # a handful of rows, small groups with zero points, K not a multiple of the tile
        dict(name="w4_five_rows", op="w4", M=5, N=11008, K=2880, group=32, zeros=True),
        # one token through a wide 4-bit block
        dict(name="w4ffn_one_token", op="w4ffn", M=1, H=5120, I=25600, group=128, zeros=False, act="silu"),
        # a decode batch through a 4-bit block
        dict(name="w4ffn_decode_32", op="w4ffn", M=32, H=4096, I=11008, group=64, zeros=True, act="silu"),
        # gradients of many small adapter matrices, fp32
        dict(name="clip_adapters", op="clip", layers=56, H=2880, I=2880, r=16, dtype="float32", bound=1.0),
        # gradients of a stack of dense blocks, bf16, odd-sized vectors among them
        dict(name="clip_blocks", op="clip", layers=4, H=4096, I=11008, r=0, dtype="bfloat16", bound=1.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["ffn", "train", "w4", "w4ffn", "clip"])
    if op == "ffn":
        return dict(op=op, T=_log(rng, 1, 2047), H=_log(rng, 256, 5120, 8), I=_log(rng, 512, 25600, 8),
                    act=rng.choice(["silu", "gelu"]))
    if op == "train":
        return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 256, 4096, 8), I=_log(rng, 256, 11008, 8),
                    act=rng.choice(["silu", "gelu"]))
    if op == "w4":
        return dict(op=op, M=_log(rng, 1, 64), N=_log(rng, 500, 25600), K=_log(rng, 512, 11008, 8),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
    if op == "w4ffn":
        return dict(op=op, M=_log(rng, 1, 64), H=_log(rng, 512, 5120, 8), I=_log(rng, 512, 25600, 8),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, act=rng.choice(["silu", "gelu"]))
    return dict(op=op, layers=_log(rng, 1, 60), H=_log(rng, 64, 4096), I=_log(rng, 64, 4096),
                r=rng.choice([8, 16, 32]), dtype=rng.choice(["float32", "bfloat16", "float16"]),
                bound=rng.choice([0.5, 1.0, 1e9]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _ffn_inputs(case, g, backward):
    T, H, I = case["T"], case["H"], case["I"]
    s = dict(x=_normal(g, (T, H), 1.0), W_gu=_normal(g, (2 * I, H), H ** -0.5),
             W_down=_normal(g, (H, I), I ** -0.5))
    if backward:
        s["dy"] = _normal(g, (T, H), 1e-2)
    return s


def _w4_inputs(g, N, K, group, zeros):
    """4-bit values two to a byte along K (the even index in the low half),
    a scale per row and group, and zero points or none."""
    G = (K + group - 1) // group
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand((N, G), generator=g, device="cuda")) * (0.2 * K ** -0.5)).to(torch.bfloat16)
    z = torch.randint(4, 12, (N, G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return dict(q=q, scales=scales, zeros=z, N=N, K=K, group=group)


def _clip_sizes(case):
    """Shapes of one program's gradients: adapters' A and B of both
    projections (r > 0), or a block's three matrices and an odd-sized vector."""
    H, I, r = case["H"], case["I"], case["r"]
    one = [(r, H), (2 * I, r), (r, I), (H, r)] if r else [(2 * I, H), (H, I), (H + 1,)]
    return [s for _ in range(case["layers"]) for s in one]


def _flat_views(shapes, dtype):
    """Tensors that lie in one flat buffer, each on a 16-byte boundary."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    offs, n = [], 0
    for s in shapes:
        offs.append(n)
        n += (math.prod(s) + per - 1) // per * per
    flat = torch.zeros(n, dtype=dtype, device="cuda")
    return flat, [flat[o:o + math.prod(s)].view(s) for o, s in zip(offs, shapes)]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("ffn", "train"):
        st.update(_ffn_inputs(case, g, op == "train"))
        if own:
            import lora_moe_amd as lm
            st["shape"] = lm.make_ffn_shape(case["T"], case["H"], case["I"], act=case["act"])
            st["ws"] = lm.alloc_ffn_workspace(st["shape"])
        return st
    if op in ("w4", "w4ffn"):
        K = case["K"] if op == "w4" else case["H"]
        st["x"] = _normal(g, (case["M"], K), 1.0)
        if op == "w4":
            parts = [("w", case["N"], K)]
        else:
            parts = [("gate", case["I"], K), ("up", case["I"], K), ("down", case["H"], case["I"])]
        for name, N, k in parts:
            w = _w4_inputs(g, N, k, case["group"], case["zeros"])
            if own:  # laid out once, when the weights are loaded
                import lora_moe_amd as lm
                w = lm.moe_lora_w4_pack(w["q"], w["scales"], w["zeros"], group=w["group"])
            st[name] = w
        if own and op == "w4ffn":
            st["ws"] = lm.alloc_w4_ffn_workspace(case["M"], case["I"])
        return st
    dtype = getattr(torch, case["dtype"])
    shapes = _clip_sizes(case)
    flat, grads = _flat_views(shapes, dtype)
    for t in grads:
        t.copy_(torch.randn(t.shape, generator=g, device="cuda") * (2.6 / math.sqrt(flat.numel())))
    out_flat, outs = _flat_views(shapes, dtype)
    st.update(grads=grads, flat_in=flat, outs=outs, flat=out_flat)
    if own:
        import lora_moe_amd as lm
        st["set"] = lm.GradSet(grads, out=outs)
    return st


# ------------------------------------------------------------------ one pass

def _act(g, kind):
    """act(g) and its derivative, in g's precision."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(GELU_C * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * GELU_C * (1.0 + 3 * 0.044715 * g * g))


def _dequant(w):
    q = torch.stack((w["q"] & 15, w["q"] >> 4), dim=2).reshape(w["N"], w["K"]).float()
    col = torch.arange(w["K"], device=q.device) // w["group"]
    z = w["zeros"].float()[:, col] if w["zeros"] is not None else 8.0
    return (q - z) * w["scales"].float()[:, col]


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("ffn", "train"):
        I = case["I"]
        x, W_gu, W_down = st["x"].float(), st["W_gu"].float(), st["W_down"].float()
        gu = x @ W_gu.t()
        g, u = gu[:, :I], gu[:, I:]
        a, da = _act(g, case["act"])
        h = a * u
        y = (h @ W_down.t()).bfloat16()
        if op == "ffn":
            return y
        dy = st["dy"].float()
        dh = dy @ W_down
        dgu = torch.cat((dh * u * da, dh * a), dim=1)
        return dict(y=y, dx=(dgu @ W_gu).bfloat16(), dW_gu=(dgu.t() @ x).bfloat16(),
                    dW_down=(dy.t() @ h).bfloat16())
    if op == "w4":
        return (st["x"].float() @ _dequant(st["w"]).t()).bfloat16()
    if op == "w4ffn":
        x = st["x"].float()
        a, _ = _act(x @ _dequant(st["gate"]).t(), case["act"])
        h = a * (x @ _dequant(st["up"]).t())
        return (h @ _dequant(st["down"]).t()).bfloat16()
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in st["grads"]:
        total = total + t.float().square().sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    coef = torch.clamp(case["bound"] / (norm + CLIP_EPS), max=1.0)
    for t, o in zip(st["grads"], st["outs"]):
        o.copy_(t.float() * coef)
    return dict(norm=norm.reshape(1), grads=st["flat"])


def _own(st):
    import lora_moe_amd as lm
    case = st["case"]
    op = case["op"]
    if op == "ffn":
        y = torch.empty_like(st["x"])
        lm.moe_lora_ffn_forward(st["shape"], st["x"], st["W_gu"], st["W_down"], st["ws"], y)
        return y
    if op == "train":
        y, dx = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        dW_gu, dW_down = torch.empty_like(st["W_gu"]), torch.empty_like(st["W_down"])
        gu = torch.empty((case["T"], 2 * case["I"]), dtype=torch.float32, device="cuda")
        lm.moe_lora_ffn_forward(st["shape"], st["x"], st["W_gu"], st["W_down"], st["ws"], y, gu=gu)
        lm.moe_lora_ffn_backward(st["shape"], st["dy"], st["x"], gu, st["W_gu"], st["W_down"], st["ws"],
                                 dx=dx, dW_gu=dW_gu, dW_down=dW_down)
        return dict(y=y, dx=dx, dW_gu=dW_gu, dW_down=dW_down)
    if op == "w4":
        y = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
        lm.moe_lora_w4_matmul(st["x"], st["w"], y)
        return y
    if op == "w4ffn":
        y = torch.empty_like(st["x"])
        lm.moe_lora_w4_ffn_forward(st["x"], st["gate"], st["up"], st["down"], st["ws"], y, act=case["act"])
        return y
    norm = torch.empty(1, dtype=torch.float32, device="cuda")
    lm.moe_lora_clip_grads(st["set"], case["bound"], norm)
    return dict(norm=norm, grads=st["flat"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floor

def _w4_bytes(N, K, group, zeros):
    G = (K + group - 1) // group
    return N * K // 2 + N * G * (3 if zeros else 2)


def work(case):
    op = case["op"]
    if op in ("ffn", "train"):
        T, H, I = case["T"], case["H"], case["I"]
        w, t = 3 * H * I * 2, T * H * 2
        if op == "ffn":
            return dict(bytes=w + 2 * t, flops=6 * T * H * I)
        return dict(bytes=2 * w + 4 * t, flops=18 * T * H * I)
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=_w4_bytes(N, K, case["group"], case["zeros"]) + 2 * M * (N + K), flops=2 * M * N * K)
    if op == "w4ffn":
        M, H, I = case["M"], case["H"], case["I"]
        b = 2 * _w4_bytes(I, H, case["group"], case["zeros"]) + _w4_bytes(H, I, case["group"], case["zeros"])
        return dict(bytes=b + 4 * M * H, flops=6 * M * H * I)
    n = sum(math.prod(s) for s in _clip_sizes(case))
    size = 4 if case["dtype"] == "float32" else 2
    return dict(bytes=2 * n * size + 4, flops=3 * n)


# ------------------------------------------------------------------ 64 bits

def _w4_exact(w):
    """The weights' values, group by group."""
    low = (w["q"] % 16).double()
    high = torch.div(w["q"], 16, rounding_mode="floor").double()
    v = torch.empty((w["N"], w["K"]), dtype=torch.float64, device=low.device)
    v[:, 0::2], v[:, 1::2] = low, high
    for j in range(w["scales"].shape[1]):
        part = v[:, j * w["group"]:(j + 1) * w["group"]]
        part -= w["zeros"][:, j:j + 1].double() if w["zeros"] is not None else 8.0
        part *= w["scales"][:, j:j + 1].double()
    return v


def _gate64(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="tanh")


def exact(case, seed):
    """The outputs in 64 bits, gradients by differentiating the definition."""
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op in ("ffn", "train"):
        I = case["I"]
        want = op == "train"
        x, W_gu, W_down = (st[k].double().requires_grad_(want) for k in ("x", "W_gu", "W_down"))
        with torch.set_grad_enabled(want):
            both = torch.nn.functional.linear(x, W_gu)
            h = _gate64(both[:, :I], case["act"]) * both[:, I:]
            y = torch.nn.functional.linear(h, W_down)
        if not want:
            return y
        dx, dW_gu, dW_down = torch.autograd.grad(y, (x, W_gu, W_down), st["dy"].double())
        return dict(y=y.detach(), dx=dx, dW_gu=dW_gu, dW_down=dW_down)
    if op == "w4":
        return st["x"].double() @ _w4_exact(st["w"]).t()
    if op == "w4ffn":
        x = st["x"].double()
        h = _gate64(x @ _w4_exact(st["gate"]).t(), case["act"]) * (x @ _w4_exact(st["up"]).t())
        return h @ _w4_exact(st["down"]).t()
    # the gaps between the tensors hold zeros: the flat buffer has the same norm
    flat = st["flat_in"].double()
    norm = torch.linalg.vector_norm(flat).reshape(1)
    c = min(1.0, case["bound"] / (float(norm) + CLIP_EPS))
    return dict(norm=norm, grads=flat.mul_(c))

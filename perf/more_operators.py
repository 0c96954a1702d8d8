"""What multi-adapter serving and fine-tuning need beside the MoE-LoRA layer, as
cases that can be timed and compared:

  proj        a shared projection with the low-rank adapters of many requests, forward
  proj_train  the same forward and backward: y, dx and the adapters' gradients
  sort        tokens sorted by expert, and the experts' rows back with the router's weights
  sort_train  the same with its gradients, the router's logits among them
  route_grad  the gradient of the router's logits alone

``run`` computes them in plain torch operations in 32 bits, or, with ``own``
set, through the library's entry points.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one request through an attention projection: the weight stream
        dict(name="proj_one_token", op="proj", T=1, K=4096, N=4096, L=8, r=16, requests=1, none=0.0),
        # a decode batch, every request with an adapter of its own choice
        dict(name="proj_decode_32", op="proj", T=32, K=4096, N=11008, L=16, r=32, requests=32, none=0.1),
        # a large decode batch over many adapters; odd token count, K and N unlike
        dict(name="proj_decode_201", op="proj", T=201, K=2880, N=5120, L=32, r=16, requests=201, none=0.0),
        # a prefill of several long requests
        dict(name="proj_prefill", op="proj", T=8192, K=7168, N=7168, L=8, r=64, requests=12, none=0.2),
        # a test model's micro-batch: what launches and latency cost
        dict(name="proj_train_small", op="proj_train", T=130, K=256, N=512, L=4, r=8, requests=5, none=0.0),
        # ragged sizes, several adapters trained in one batch, some tokens without one
        dict(name="proj_train_ragged", op="proj_train", T=1001, K=2880, N=2880, L=16, r=32, requests=23, none=0.1),
        # a full micro-batch of one base model under several adapters
        dict(name="proj_train_large", op="proj_train", T=8192, K=4096, N=4096, L=8, r=16, requests=16, none=0.0),
        # a decode batch to its experts and back
        dict(name="sort_decode_16", op="sort", T=16, H=4096, E=8, topk=2, dtype="bfloat16", spread=0.0),
        # a prefill over many experts, unevenly loaded
        dict(name="sort_prefill", op="sort", T=8192, H=7168, E=256, topk=8, dtype="bfloat16", spread=2.0),
        # a training micro-batch of odd size in half precision
        dict(name="sort_train_ragged", op="sort_train", T=1001, H=2880, E=32, topk=4, dtype="float16", spread=1.0),
        # a full training micro-batch with 32-bit rows
        dict(name="sort_train_large", op="sort_train", T=4096, H=2048, E=128, topk=8, dtype="float32", spread=0.5),
        # the router of a long micro-batch
        dict(name="route_grad", op="route_grad", T=8192, E=256, topk=8, spread=1.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["proj", "proj_train", "sort", "sort_train", "route_grad"])
    if op in ("proj", "proj_train"):
        wide = 7168 if op == "proj" else 4096
        T, r = _log(rng, 1, 8192), rng.choice([8, 16, 24, 32, 64])
        return dict(op=op, T=T, K=_log(rng, 256, wide, 8), N=_log(rng, 256, wide, 8),
                    L=_log(rng, 1, min(64, 2048 // r)), r=r,
                    requests=T if T <= 256 and rng.random() < 0.7 else _log(rng, 1, max(1, min(T, 64))),
                    none=rng.choice([0.0, 0.1, 0.5]))
    if op == "route_grad":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, topk=rng.randint(1, min(8, E)), spread=rng.choice([0.5, 2.0]))
    E = _log(rng, 4, 256)
    big = (8192, 7168) if op == "sort" else (4096, 2048)
    return dict(op=op, T=_log(rng, 1, big[0]), H=_log(rng, 256, big[1], 8), E=E, topk=rng.randint(1, min(8, E)),
                dtype=rng.choice(["bfloat16", "bfloat16", "float16"] + ["float32"] * (op == "sort_train")),
                spread=rng.choice([0.0, 1.0, 2.0]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _adapter_ids(g, case):
    """Tokens in runs, one for each request (a decode batch: one token each);
    every request takes an adapter at random, or none (-1)."""
    T, R = case["T"], case["requests"]
    cuts = torch.sort(torch.randint(0, T, (R - 1,), generator=g, device="cuda"))[0]
    request = torch.arange(T, device="cuda") if R >= T else torch.searchsorted(cuts, torch.arange(T, device="cuda"),
                                                                               right=True)
    adapter = torch.randint(0, case["L"], (max(R, T),), generator=g, device="cuda")
    without = torch.rand(adapter.shape, generator=g, device="cuda") < case["none"]
    return torch.where(without, -1, adapter)[request].int()


def _logits(g, case):
    T, E = case["T"], case["E"]
    return (torch.randn((T, E), generator=g, device="cuda")
            + case["spread"] * torch.randn((1, E), generator=g, device="cuda"))


def _routed(g, case):
    """Each token's experts by descending logit, and the softmax over those."""
    v, ids = torch.topk(_logits(g, case), case["topk"], dim=1)
    return ids.int().contiguous(), torch.softmax(v, dim=1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("proj", "proj_train"):
        T, K, N, L, r = (case[k] for k in ("T", "K", "N", "L", "r"))
        st.update(x=_normal(g, (T, K), 1.0), W=_normal(g, (N, K), K ** -0.5), A=_normal(g, (L, r, K), K ** -0.5),
                  B=_normal(g, (L, N, r), 0.5 * r ** -0.5), ids=_adapter_ids(g, case),
                  # alpha / r of each adapter
                  scales=torch.tensor([0.5, 1.0, 2.0], device="cuda")[torch.arange(L, device="cuda") % 3])
        if op == "proj_train":
            st["dy"] = _normal(g, (T, N), 1e-2)
        if own:
            import lora_moe_amd as lm
            st["shape"] = lm.make_proj_shape(T, K, N, L, r)
            st["ws"] = lm.alloc_proj_workspace(st["shape"], backward=op == "proj_train")
        return st
    st["ids"], st["weights"] = _routed(g, case)
    if op == "route_grad":
        st["dweights"] = torch.randn(st["weights"].shape, generator=g, device="cuda") * 1e-2
        if own:
            import lora_moe_amd as lm
            st["route"] = lm.make_shape(case["T"], 8, 8, case["E"], case["topk"], 1, 8)
        return st
    T, H, P, dtype = case["T"], case["H"], case["T"] * case["topk"], getattr(torch, case["dtype"])
    st["x"] = _normal(g, (T, H), 1.0, dtype)
    st["d"] = _normal(g, (P, H), 1.0, dtype)       # the experts' outputs, sorted rows
    if op == "sort_train":
        st["dy"] = _normal(g, (T, H), 1e-2, dtype)
        st["dxs"] = _normal(g, (P, H), 1e-2, dtype)  # gradients of the sorted rows, from the experts
    if own:
        import lora_moe_amd as lm
        st["shape"] = lm.make_sort_shape(T, H, case["E"], case["topk"], dtype)
        st["ws"] = lm.alloc_sort_workspace(st["shape"])
        if op == "sort_train":
            st["route"] = lm.make_shape(T, H, 8, case["E"], case["topk"], 1, 8)
    return st


# ------------------------------------------------------------------ one pass

def _own_columns(st):
    """[T, L r]: 1 in the columns of a token's own adapter, and the scale of
    each token's."""
    case = st["case"]
    ids = st["ids"].long()
    column = torch.arange(case["L"] * case["r"], device="cuda") // case["r"]
    s = torch.where(ids >= 0, st["scales"][ids.clamp(min=0)], 0.0)
    return (column[None, :] == ids[:, None]).float(), s[:, None]


def _plain_proj(st):
    case = st["case"]
    L, r, K, N = case["L"], case["r"], case["K"], case["N"]
    x, W = st["x"].float(), st["W"].float()
    A = st["A"].float().reshape(L * r, K)
    B = st["B"].float().transpose(1, 2).reshape(L * r, N)
    mine, s = _own_columns(st)
    z = (x @ A.t()) * mine * s
    y = (x @ W.t() + z @ B).bfloat16()
    if case["op"] == "proj":
        return y
    dy = st["dy"].float()
    u = (dy @ B.t()) * mine * s
    dA = (u.t() @ x).reshape(L, r, K).bfloat16()
    dB = (z.t() @ dy).reshape(L, r, N).transpose(1, 2).contiguous().bfloat16()
    return dict(y=y, dx=(dy @ W + u @ A).bfloat16(), dA=dA, dB=dB)


def _plain_route_grad(ids, w, dw, E):
    g = w * (dw - (w * dw).sum(dim=1, keepdim=True))
    return torch.zeros((w.shape[0], E), device="cuda").scatter_(1, ids.long(), g)


def _plain_sort(st):
    case = st["case"]
    T, H, E, k, dtype = case["T"], case["H"], case["E"], case["topk"], getattr(torch, case["dtype"])
    expert, pair = torch.sort(st["ids"].reshape(-1), stable=True)
    edges = torch.arange(E + 1, device="cuda", dtype=torch.int32)
    out = dict(expert_off=torch.searchsorted(expert, edges).int())
    row = torch.empty(T * k, dtype=torch.int64, device="cuda")
    row[pair] = torch.arange(T * k, device="cuda")
    token = pair // k
    out["row_of_pair"] = row.reshape(T, k).int()
    out["rows"] = st["x"].float()[token].to(dtype)
    w = st["weights"]
    mine = st["d"].float()[row].reshape(T, k, H)
    out["y"] = (mine * w[:, :, None]).sum(dim=1).to(dtype)
    if case["op"] == "sort":
        return out
    dy = st["dy"].float()
    out["dd"] = (dy[token] * w.reshape(-1)[pair][:, None]).to(dtype)
    dw = (mine * dy[:, None, :]).sum(dim=2)
    out["dweights"] = dw
    out["dx"] = st["dxs"].float()[row].reshape(T, k, H).sum(dim=1).to(dtype)
    out["dlogits"] = _plain_route_grad(st["ids"], w, dw, E)
    return out


def _own(st):
    import lora_moe_amd as lm
    case = st["case"]
    op = case["op"]
    if op == "proj":
        y = torch.empty((case["T"], case["N"]), dtype=torch.bfloat16, device="cuda")
        lm.moe_lora_proj_forward(st["shape"], st["x"], st["ids"], st["W"], st["A"], st["B"], st["ws"], y,
                                 scales=st["scales"])
        return y
    if op == "proj_train":
        y, dx = torch.empty_like(st["dy"]), torch.empty_like(st["x"])
        dA, dB = torch.empty_like(st["A"]), torch.empty_like(st["B"])
        z = torch.empty((case["T"], case["r"]), dtype=torch.float32, device="cuda")
        lm.moe_lora_proj_forward(st["shape"], st["x"], st["ids"], st["W"], st["A"], st["B"], st["ws"], y, z=z,
                                 scales=st["scales"])
        lm.moe_lora_proj_backward(st["shape"], st["dy"], st["x"], st["ids"], z, st["W"], st["A"], st["B"], st["ws"],
                                  dx=dx, dA=dA, dB=dB, scales=st["scales"])
        return dict(y=y, dx=dx, dA=dA, dB=dB)
    if op == "route_grad":
        dlogits = torch.empty((case["T"], case["E"]), device="cuda")
        lm.moe_lora_route_backward(st["route"], st["ids"], st["weights"], st["dweights"], dlogits)
        return dlogits
    out = dict(rows=torch.empty_like(st["d"]), y=torch.empty_like(st["x"]),
               expert_off=torch.empty(case["E"] + 1, dtype=torch.int32, device="cuda"),
               row_of_pair=torch.empty_like(st["ids"]))
    lm.moe_lora_sort(st["shape"], st["ids"], st["x"], st["ws"], out["rows"], out["expert_off"], out["row_of_pair"])
    lm.moe_lora_unsort(st["shape"], st["d"], out["row_of_pair"], out["y"], weights=st["weights"])
    if op == "sort":
        return out
    out.update(dd=torch.empty_like(st["d"]), dweights=torch.empty_like(st["weights"]), dx=torch.empty_like(st["x"]),
               dlogits=torch.empty((case["T"], case["E"]), device="cuda"))
    lm.moe_lora_unsort_backward(st["shape"], st["dy"], st["d"], out["row_of_pair"], out["dd"],
                                weights=st["weights"], dweights=out["dweights"])
    lm.moe_lora_sort_backward(st["shape"], st["dxs"], out["row_of_pair"], out["dx"])
    lm.moe_lora_route_backward(st["route"], st["ids"], st["weights"], out["dweights"], out["dlogits"])
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("proj", "proj_train"):
        return _plain_proj(state)
    if op == "route_grad":
        return _plain_route_grad(state["ids"], state["weights"], state["dweights"], state["case"]["E"])
    return _plain_sort(state)


# ------------------------------------------------------------------ floor

def work(case):
    op, T = case["op"], case["T"]
    if op in ("proj", "proj_train"):
        K, N, r = case["K"], case["N"], case["r"]
        met = min(case["L"], case["requests"])  # adapters that are met, at most
        b = 2 * (T * K + T * N + N * K + met * r * (K + N)) + 4 * T
        f = 2 * T * (K * N + r * (K + N))
        if op == "proj_train":
            b += 2 * (T * K + T * N + case["L"] * r * (K + N))
            f += 2 * T * (K * N + 2 * r * (K + N))
        return dict(bytes=b, flops=f)
    E, k = case["E"], case["topk"]
    route = T * E * 4 + T * k * 12
    if op == "route_grad":
        return dict(bytes=route, flops=4 * T * k)
    row = case["H"] * (4 if case["dtype"] == "float32" else 2)
    b = (2 * T + 2 * T * k) * row + T * k * 12 + 4 * E
    f = 2 * T * k * case["H"]
    if op == "sort_train":
        # dy in, dx out; the experts' rows again, their gradients out, the sorted rows' gradients in (the rows meet
        # both the weights and dy: read once where a pass over them did both)
        b += (2 * T + 2 * T * k) * row + route
        f += 4 * T * k * case["H"]
    return dict(bytes=b, flops=f)


# ------------------------------------------------------------------ 64 bits

def _exact_proj(st):
    case = st["case"]
    train = case["op"] == "proj_train"
    x, W, A, B = (st[k].double().requires_grad_(train) for k in ("x", "W", "A", "B"))
    with torch.set_grad_enabled(train):
        y = torch.nn.functional.linear(x, W.detach())
        for l in range(case["L"]):
            at = torch.nonzero(st["ids"] == l).flatten()
            if at.numel():
                y = y.index_add(0, at, (x[at] @ A[l].T @ B[l].T) * float(st["scales"][l]))
    if not train:
        return y
    dx, dA, dB = torch.autograd.grad(y, (x, A, B), st["dy"].double(), allow_unused=True)
    return dict(y=y.detach(), dx=dx, dA=torch.zeros_like(A) if dA is None else dA,
                dB=torch.zeros_like(B) if dB is None else dB)


def _exact_route(ids, w, dw, E):
    """By the softmax's Jacobian over the chosen logits."""
    w, dw = w.double(), dw.double()
    J = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    d = torch.zeros((w.shape[0], E), dtype=torch.float64, device=w.device)
    return d.index_put_((torch.arange(w.shape[0], device=w.device)[:, None], ids.long()), (J @ dw[:, :, None])[:, :, 0],
                        accumulate=True)


def _exact_sort(st):
    case = st["case"]
    T, H, E, k = case["T"], case["H"], case["E"], case["topk"]
    flat = st["ids"].reshape(-1)
    hot = (flat[:, None] == torch.arange(E, device="cuda")[None, :]).int()
    ends = torch.cumsum(hot.sum(dim=0), 0)
    off = torch.cat((ends.new_zeros(1), ends))
    rank = (torch.cumsum(hot, 0) * hot).sum(dim=1) - 1
    row = off[flat.long()] + rank
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    w, train = st["weights"].double().reshape(-1, 1), case["op"] == "sort_train"
    rows = torch.zeros((T * k, H), dtype=torch.float64, device="cuda").index_copy_(0, row, st["x"].double()[token])
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    d = st["d"].double()
    for j in range(k):
        y.addcmul_(d[row[j::k]], w[j::k])
    out = dict(expert_off=off.int(), row_of_pair=row.reshape(T, k).int(), rows=rows, y=y)
    if train:
        dy = st["dy"].double()
        out["dd"] = torch.zeros_like(rows).index_copy_(0, row, dy[token] * w)
        out["dweights"] = torch.linalg.vecdot(d[row], dy[token]).reshape(T, k)
        out["dx"] = torch.zeros_like(y).index_add_(0, token, st["dxs"].double()[row])
        out["dlogits"] = _exact_route(st["ids"], st["weights"], out["dweights"], E)
    return out


def exact(case, seed):
    """The outputs in 64 bits, the projection's gradients by differentiating
    its definition."""
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] in ("proj", "proj_train"):
        return _exact_proj(st)
    if case["op"] == "route_grad":
        return _exact_route(st["ids"], st["weights"], st["dweights"], case["E"])
    return _exact_sort(st)

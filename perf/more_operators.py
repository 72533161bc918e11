"""Cases of the operators that train and adapt expert layers in bf16: grouped products and their weights'
gradients, SwiGLU and its gradient, and low-rank adapters of many requests.

  product    y[m] = a[m] W_e^T (or a[m] W_e, the gradient by the input), the rows of `a` grouped by
             expert: rows offsets[e] .. offsets[e + 1] take expert e's weights, rows of no expert give 0
  weights    dW_e = sum over expert e's rows of dy[m]^T a[m] (0 for an expert without rows)
  swiglu     h = silu(g) * u of rows [g | u], and the gradient by both
  lora       out[t] = base[t] + v B_e^T with v = scale_e x[t] A_e^T, e the adapter of token t; tokens of
             no adapter keep base.  The tokens sorted by adapter (a plan) are kept by the program
             for all of its layers
  lora_back  the gradients: dv = scale_e dy[t] B_e, dx[t] = base[t] + dv A_e, dA_e = sum dv^T x[t],
             dB_e = sum dy[t]^T v
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token's eight experts of the routed layer (128 experts, 2048 -> gate and up of 768)
        {"name": "product_token", "op": "product", "tokens": 1, "top_k": 8, "experts": 128, "n": 1536, "k": 2048, "back": False, "out": "bf16", "dropped": 0.0},
        # a batch of 256 tokens through the same layer: about 16 rows an expert, unevenly
        {"name": "product_batch", "op": "product", "tokens": 256, "top_k": 8, "experts": 128, "n": 1536, "k": 2048, "back": False, "out": "bf16", "dropped": 0.0},
        # a training step's 4096 tokens: about 256 rows an expert, unevenly
        {"name": "product_prompt", "op": "product", "tokens": 4096, "top_k": 8, "experts": 128, "n": 1536, "k": 2048, "back": False, "out": "bf16", "dropped": 0.0},
        # gradient by the input of a small uneven batch of odd sizes, some pairs without an expert
        {"name": "product_back_ragged", "op": "product", "tokens": 465, "top_k": 4, "experts": 27, "n": 2056, "k": 1032, "back": True, "out": "fp32", "dropped": 0.05},
        # the weights' gradients of a small uneven batch, kept in fp32
        {"name": "weights_ragged", "op": "weights", "tokens": 465, "top_k": 4, "experts": 27, "n": 1032, "k": 2056, "out": "fp32", "dropped": 0.05},
        # the weights' gradients of the training step's gate and up projections
        {"name": "weights_prompt", "op": "weights", "tokens": 4096, "top_k": 8, "experts": 128, "n": 1536, "k": 2048, "out": "bf16", "dropped": 0.0},
        # SwiGLU between the training step's products
        {"name": "swiglu_prompt", "op": "swiglu", "rows": 32768, "i": 768, "type": "bf16", "back": False},
        # its gradient for a small batch of an odd width
        {"name": "swiglu_back_ragged", "op": "swiglu", "rows": 1859, "i": 1021, "type": "fp32", "back": True},
        # decoding requests, each with an adapter of its own, beside the 4096 -> 11008 projection
        {"name": "lora_batch", "op": "lora", "tokens": 61, "adapters": 48, "rank": 16, "n": 11008, "k": 4096, "out": "bf16", "packed": False, "none": 0.1},
        # prompts of eight adapters packed one after another beside the same projection
        {"name": "lora_prompt", "op": "lora", "tokens": 2048, "adapters": 8, "rank": 64, "n": 11008, "k": 4096, "out": "bf16", "packed": True, "none": 0.0},
        # gradients of a small mixed batch of odd sizes
        {"name": "lora_back_ragged", "op": "lora_back", "tokens": 333, "adapters": 5, "rank": 24, "n": 2056, "k": 1032, "out": "fp32", "packed": False, "none": 0.1},
        # gradients of a training step's 4096 tokens, four adapters at once
        {"name": "lora_back_prompt", "op": "lora_back", "tokens": 4096, "adapters": 4, "rank": 32, "n": 11008, "k": 4096, "out": "bf16", "packed": True, "none": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "weights", "weights", "swiglu", "lora", "lora", "lora_back"])
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "swiglu":
        rows, i = _log(rng, 1, 32768), _log(rng, 32, 11008)
        while rows * i > 32768 * 768:
            rows //= 2
        return {"op": op, "rows": max(1, rows), "i": i, "type": out, "back": rng.random() < 0.5}
    n, k = 8 * _log(rng, 8, 1376), 8 * _log(rng, 8, 1376)
    if op in ("product", "weights"):
        experts = _log(rng, 1, 128)
        while experts * n * k > 128 * 1536 * 2048 // (2 if out == "fp32" else 1):
            experts = max(1, experts // 2)
        top_k = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, 4096)
        tokens = max(1, min(tokens, int(1e11 / (top_k * n * k)), int(3e8 / (top_k * (n + k)) / (2 if out == "fp32" else 1))))
        case = {"op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "n": n, "k": k, "out": out, "dropped": rng.choice([0.0, 0.0, 0.1])}
        if op == "product":
            case["back"] = rng.random() < 0.5
        return case
    tokens, adapters, rank = _log(rng, 1, 4096), _log(rng, 1, 64), 8 * rng.choice([1, 2, 2, 3, 4, 8, 16])
    while adapters * rank * (n + k) > 32 * 64 * 15104:
        adapters = max(1, adapters // 2)
    return {"op": op, "tokens": tokens, "adapters": adapters, "rank": rank, "n": n, "k": k, "out": out,
            "packed": rng.random() < 0.5, "none": rng.choice([0.0, 0.1, 0.3])}


# ---- inputs --------------------------------------------------------------------------------

def _activations(g, rows, cols):
    """N(0, 1) with 1 % of the columns 20 times larger, as hidden states have them."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return (x * torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.01, 20.0, 1.0)).to(torch.bfloat16)


def _gradients(g, rows, cols):
    return (torch.randn((rows, cols), generator=g, device="cuda") * 0.01).to(torch.bfloat16)


def _weights(g, *shape):
    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for e in range(shape[0]):
        w[e] = torch.randn(shape[1:], generator=g, device="cuda") * 0.02
    return w


def _ids(g, case):
    """Each token's experts: the top_k of logits N(0, 1) with a bias for each expert, so that the
    experts' loads differ; -1 for pairs that are dropped."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn((t, e), generator=g, device="cuda") + 0.4 * torch.randn((e,), generator=g, device="cuda")
    ids = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
    if case["dropped"]:
        ids[torch.rand((t, k), generator=g, device="cuda") < case["dropped"]] = -1
    return ids


def _adapters(g, case):
    """Each token's adapter: drawn for each, or sequences of uneven lengths one after another; -1 for none."""
    t, n = case["tokens"], case["adapters"]
    ids = torch.randint(0, n, (t,), generator=g, device="cuda")
    if case["packed"]:
        ids = torch.sort(ids)[0]
        ids = torch.randperm(n, generator=g, device="cuda")[ids]
    if case["none"]:
        ids = torch.where(torch.rand((t,), generator=g, device="cuda") < case["none"], -1, ids)
    return ids.to(torch.int32).view(t, 1)


def _sort(ids, groups):
    """row_slot [T k] (-1 past the last group), slot_row [T, k] (-1: no group), offsets [groups + 1]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    sorted_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(sorted_key, torch.arange(groups + 1, device=ids.device))
    row = torch.arange(flat.numel(), device=ids.device)
    row_slot = torch.where(sorted_key < groups, order, -1)
    slot_row = torch.empty_like(row)
    slot_row[order] = torch.where(sorted_key < groups, row, -1)
    return row_slot.to(torch.int32), slot_row.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    kind = DT[case.get("out", "bf16")]
    if op == "swiglu":
        rows, i, kind = case["rows"], case["i"], DT[case["type"]]
        s["gu"] = (torch.randn((rows, 2 * i), generator=g, device="cuda") * 2.0).to(kind)
        if case["back"]:
            s["dh"] = (torch.randn((rows, i), generator=g, device="cuda") * 0.01).to(kind)
        s["out"] = torch.empty((rows, 2 * i if case["back"] else i), dtype=kind, device="cuda")
        return s
    n, k = case["n"], case["k"]
    if op in ("product", "weights"):
        rows, experts = case["tokens"] * case["top_k"], case["experts"]
        s["offsets"] = _sort(_ids(g, case), experts)[2]
        s["most"] = max(1, int(s["offsets"].diff().max()))
        if op == "weights":
            s["a"], s["dy"] = _activations(g, rows, k), _gradients(g, rows, n)
            s["out"] = torch.empty((experts, n, k), dtype=kind, device="cuda")
        else:
            s["a"] = _gradients(g, rows, k) if case["back"] else _activations(g, rows, k)
            s["w"] = _weights(g, experts, k, n) if case["back"] else _weights(g, experts, n, k)
            s["out"] = torch.empty((rows, n), dtype=kind, device="cuda")
        return s
    tokens, adapters, rank = case["tokens"], case["adapters"], case["rank"]
    s["plan"] = _sort(_adapters(g, case), adapters)
    s["most"] = max(1, int(s["plan"][2].diff().max()))
    s["x"] = _activations(g, tokens, k)
    s["A"], s["B"] = _weights(g, adapters, rank, k), _weights(g, adapters, n, rank)
    s["scale"] = 2.0 ** torch.randint(-1, 2, (adapters,), generator=g, device="cuda").float()
    if op == "lora":
        s["base"] = torch.randn((tokens, n), generator=g, device="cuda").to(kind)
        s["out"] = torch.empty_like(s["base"])
        s["v"] = torch.empty((tokens, rank), device="cuda")
        return s
    s["dy"] = _gradients(g, tokens, n)
    s["v"] = torch.randn((tokens, rank), generator=g, device="cuda")
    s["v"][int(s["plan"][2][-1]):] = 0.0
    s["base"] = (torch.randn((tokens, k), generator=g, device="cuda") * 0.01).to(kind)
    s["dx"] = torch.empty_like(s["base"])
    s["dA"], s["dB"] = torch.empty_like(s["A"], dtype=kind), torch.empty_like(s["B"], dtype=kind)
    return s


# ---- plain forms ---------------------------------------------------------------------------

def _places(offsets, rows, groups, most):
    """Row -> its place in [groups, most] (one more place for rows of no group), and whether it has one."""
    row = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long(), row, right=True)
    some = e.clamp(max=groups - 1)
    return torch.where(e < groups, some * most + row - offsets.long()[some], groups * most), (e < groups)[:, None], some


def _padded(x, place, some, groups, most):
    """Rows [rows, c] at their places [groups, most, c] in fp32, zeros between them."""
    p = torch.zeros((groups * most + 1, x.shape[1]), device=x.device)
    p[place] = torch.where(some, x.float(), 0.0)
    return p[:-1].view(groups, most, -1)


def _grouped(x, w, offsets, most):
    """x [rows, k] times w [groups, k, n] of each row's group, fp32; 0 for rows of none."""
    groups, k, n = w.shape
    place, some, e = _places(offsets, x.shape[0], groups, most)
    if x.shape[0] <= groups:  # few rows: each takes its own group's weights
        return torch.bmm(x.float().view(-1, 1, k), w[e].float()).view(-1, n) * some
    y = torch.zeros((groups * most + 1, n), device=x.device)
    y[:-1] = torch.bmm(_padded(x, place, some, groups, most), w.float()).view(-1, n)
    return y[place]


def _grouped_outer(a, b, offsets, most):
    """sum over each group's rows of a[row]^T b[row]: [groups, a's columns, b's columns], fp32."""
    groups = offsets.numel() - 1
    place, some, _ = _places(offsets, a.shape[0], groups, most)
    return torch.bmm(_padded(a, place, some, groups, most).transpose(1, 2), _padded(b, place, some, groups, most))


def _row_scale(scale, offsets, rows):
    row = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long(), row, right=True)
    return scale[e.clamp(max=scale.numel() - 1)][:, None]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from quantized_ffn_gb300 import zffn
        if op == "product":
            return zffn.bf16_matmul(state["a"], state["w"], offsets=state["offsets"], transposed=case["back"], y=state["out"])
        if op == "weights":
            return zffn.bf16_matmul_grad_w(state["dy"], state["a"], offsets=state["offsets"], dw=state["out"])
        if op == "swiglu":
            if case["back"]:
                return zffn.swiglu_grad(state["dh"], state["gu"], dgu=state["out"])
            return zffn.swiglu(state["gu"], h=state["out"])
        plan = zffn.MoePlan(*state["plan"])
        if op == "lora":
            return zffn.lora_add(state["x"], state["A"], state["B"], plan, scale=state["scale"], base=state["base"],
                                 out=state["out"], v=state["v"])
        return zffn.lora_grad(state["dy"], state["x"], state["v"], state["A"], state["B"], plan, scale=state["scale"],
                              base=state["base"], dx=state["dx"], dA=state["dA"], dB=state["dB"])
    if op == "product":
        w = state["w"] if case["back"] else state["w"].transpose(1, 2)
        return _grouped(state["a"], w, state["offsets"], state["most"]).to(state["out"].dtype)
    if op == "weights":
        return _grouped_outer(state["dy"], state["a"], state["offsets"], state["most"]).to(state["out"].dtype)
    if op == "swiglu":
        g, u = state["gu"].float().chunk(2, 1)
        sig = 1.0 / (1.0 + torch.exp(-g))
        if not case["back"]:
            return (g * sig * u).to(state["out"].dtype)
        dh = state["dh"].float()
        return torch.cat((dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig), 1).to(state["out"].dtype)
    row_slot, slot_row, offsets = state["plan"]
    most, tokens = state["most"], case["tokens"]
    token, place = row_slot.long().clamp(min=0), slot_row.view(-1).long()
    some, has = (row_slot >= 0)[:, None], (place >= 0)[:, None]
    scale = _row_scale(state["scale"], offsets, tokens)

    def back(rows):
        return torch.where(has, rows[place.clamp(min=0)], 0.0)

    xs = torch.where(some, state["x"][token], 0.0)
    if op == "lora":
        v = _grouped(xs, state["A"].transpose(1, 2), offsets, most) * scale
        out = state["base"].float() + back(_grouped(v, state["B"].transpose(1, 2), offsets, most))
        return out.to(state["out"].dtype), v
    dys = torch.where(some, state["dy"][token], 0.0)
    dv = _grouped(dys, state["B"], offsets, most) * scale
    dx = state["base"].float() + back(_grouped(dv, state["A"], offsets, most))
    dA, dB = _grouped_outer(dv, xs, offsets, most), _grouped_outer(dys, state["v"], offsets, most)
    return dx.to(state["dx"].dtype), dA.to(state["dA"].dtype), dB.to(state["dB"].dtype)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "swiglu":
        each = case["rows"] * case["i"]
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": each * size * (5 if case["back"] else 3), "flops": each * (10 if case["back"] else 5)}
    n, k, size = case["n"], case["k"], 2 if case["out"] == "bf16" else 4
    if op in ("product", "weights"):
        m, e = case["tokens"] * case["top_k"], case["experts"]
        if op == "weights":
            return {"bytes": 2 * m * (n + k) + e * n * k * size, "flops": 2 * m * n * k}
        return {"bytes": 2 * m * k + 2 * min(e, m) * n * k + m * n * size, "flops": 2 * m * n * k}
    t, r, e = case["tokens"], case["rank"], min(case["adapters"], case["tokens"])
    if op == "lora":
        return {"bytes": 2 * t * k + 2 * e * r * (n + k) + 2 * t * n * size + 4 * t * r, "flops": 2 * t * r * (n + k)}
    return {"bytes": 2 * t * (n + k) + 2 * e * r * (n + k) + 4 * t * r + 2 * t * k * size + case["adapters"] * r * (n + k) * size,
            "flops": 4 * t * r * (n + k)}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "swiglu":
        g, u = s["gu"][:, :case["i"]].double(), s["gu"][:, case["i"]:].double()
        if not case["back"]:
            return torch.sigmoid(g) * g * u
        dh, sig = s["dh"].double(), torch.sigmoid(g)
        return torch.hstack((dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * (g * sig)))
    if op in ("product", "weights"):
        cut = s["offsets"].tolist()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            rows = slice(cut[e], cut[e + 1])
            if cut[e] == cut[e + 1]:
                continue
            a = s["a"][rows].double()
            if op == "weights":
                out[e] = s["dy"][rows].double().T @ a
            else:
                w = s["w"][e].double()
                out[rows] = a @ (w if case["back"] else w.T)
        return out
    row_slot, cut = s["plan"][0].long(), s["plan"][2].tolist()
    x, A, B = s["x"].double(), s["A"].double(), s["B"].double()
    if op == "lora":
        out, v = s["base"].double(), torch.zeros((case["tokens"], case["rank"]), dtype=torch.float64, device="cuda")
        for e in range(case["adapters"]):
            t = row_slot[cut[e]:cut[e + 1]]
            v[cut[e]:cut[e + 1]] = s["scale"][e].double() * (x[t] @ A[e].T)
            out[t] += v[cut[e]:cut[e + 1]] @ B[e].T
        return out, v
    dy, v, dx = s["dy"].double(), s["v"].double(), s["base"].double()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for e in range(case["adapters"]):
        t = row_slot[cut[e]:cut[e + 1]]
        dv = s["scale"][e].double() * (dy[t] @ B[e])
        dx[t] += dv @ A[e]
        dA[e] = dv.T @ x[t]
        dB[e] = dy[t].T @ v[cut[e]:cut[e + 1]]
    return dx, dA, dB

"""Cases of the 8-bit expert operators: block-scaled products, their quantisation, and tokens sorted by expert.

Four operators, used one after another by a routed layer whose weights are held in
8-bit floating point (e4m3) with one fp32 scale for each block of 128:

  quantise   rows of bf16 or fp32 -> e4m3 and a power-of-two scale for each 128 columns of a
             row (activations), or for each 128 x 128 block (weights)
  product    y[m, n] = sum_k a[m, k] sa[m, k/128] w[n, k] sw[n/128, k/128], dense or with the
             rows of `a` grouped by expert
  experts    the two products of a routed layer's experts over rows sorted by expert, with
             h = quantise(silu(a Wg^T) * (a Wu^T)) between them
  dispatch   the stable sort of (token, slot) pairs by expert, the copy of each token's row to
             its sorted places, and the weighted sum of the experts' rows back to tokens
  gradient   of the dispatch: dx; of the weighted sum: the rows' and the weights' gradients
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token through the gate matrix of the 4096 / 11008 layer: a decode step
        {"name": "product_token", "op": "product", "rows": 1, "n": 11008, "k": 4096, "experts": 0, "out": "bf16"},
        # a small batch of decoding requests on a matrix of odd sizes, last blocks cut on both axes
        {"name": "product_ragged", "op": "product", "rows": 37, "n": 2057, "k": 1040, "experts": 0, "out": "fp32"},
        # a prompt of 2048 tokens through the same gate matrix
        {"name": "product_prompt", "op": "product", "rows": 2048, "n": 11008, "k": 4096, "experts": 0, "out": "bf16"},
        # one token's eight experts of the routed layer (128 experts, 2048 / 768)
        {"name": "experts_token", "op": "experts", "tokens": 1, "top_k": 8, "experts": 128, "h": 2048, "i": 768, "dropped": 0.0},
        # a batch of 256 tokens: about 16 rows an expert, unevenly
        {"name": "experts_batch", "op": "experts", "tokens": 256, "top_k": 8, "experts": 128, "h": 2048, "i": 768, "dropped": 0.0},
        # a prompt of 4096 tokens: about 256 rows an expert, unevenly
        {"name": "experts_prompt", "op": "experts", "tokens": 4096, "top_k": 8, "experts": 128, "h": 2048, "i": 768, "dropped": 0.0},
        # a small batch before a product, last block cut
        {"name": "quantise_ragged", "op": "quantise", "rows": 37, "k": 1040, "in": "fp32", "block_rows": 1},
        # a prompt's sorted rows before the experts
        {"name": "quantise_prompt", "op": "quantise", "rows": 16384, "k": 2048, "in": "bf16", "block_rows": 1},
        # one token to its eight experts and back
        {"name": "dispatch_token", "op": "dispatch", "tokens": 1, "top_k": 8, "experts": 128, "h": 2048, "in": "bf16", "dropped": 0.0},
        # a prompt to its experts and back, some pairs without an expert (padding, dropped tokens)
        {"name": "dispatch_prompt", "op": "dispatch", "tokens": 4096, "top_k": 8, "experts": 128, "h": 2048, "in": "bf16", "dropped": 0.02},
        # gradients of a small batch of odd sizes
        {"name": "gradient_ragged", "op": "gradient", "tokens": 37, "top_k": 5, "experts": 60, "h": 1041, "in": "fp32", "dropped": 0.05},
        # gradients of a training step's 4096 tokens
        {"name": "gradient_prompt", "op": "gradient", "tokens": 4096, "top_k": 8, "experts": 128, "h": 2048, "in": "bf16", "dropped": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "experts", "experts", "quantise", "dispatch", "gradient"])
    if op == "product":
        experts = rng.choice([0, 0, 0, _log(rng, 2, 64)])
        n, k = _log(rng, 64, 11008), 16 * _log(rng, 8, 688)
        while experts * n * k > 1 << 29:
            n, k = max(64, n // 2), max(128, k // 32 * 16)
        rows = _log(rng, 1, 4096)
        rows = max(1, min(rows, int(9e10 / (n * k))))
        return {"op": op, "rows": rows, "n": n, "k": k, "experts": experts, "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "quantise":
        rows, k = _log(rng, 1, 16384), _log(rng, 64, 11008)
        while rows * k > 1 << 25:
            rows //= 2
        return {"op": op, "rows": rows, "k": k, "in": rng.choice(["bf16", "bf16", "fp32"]), "block_rows": rng.choice([1, 1, 1, 128])}
    experts = _log(rng, 2, 128)
    top_k = rng.randint(1, min(8, experts))
    tokens = _log(rng, 1, 4096)
    dropped = rng.choice([0.0, 0.0, 0.1])
    if op == "experts":
        h, i = 16 * _log(rng, 8, 256), 16 * _log(rng, 4, 128)
        while experts * h * i > 128 * 2048 * 768:
            experts = max(top_k, experts // 2)
            if experts == top_k:
                i = max(64, i // 32 * 16)
        tokens = max(1, min(tokens, int(5.1e10 / (top_k * h * i))))
        return {"op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "h": h, "i": i, "dropped": dropped}
    h = _log(rng, 64, 8192)
    tokens = max(1, min(tokens, (1 << 26) // (top_k * h)))
    return {"op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "h": h, "in": rng.choice(["bf16", "bf16", "fp32"]), "dropped": dropped}


# ---- inputs --------------------------------------------------------------------------------

def _blocks(n):
    return -(-n // BLOCK)


def _activations(g, rows, cols):
    """N(0, 1) with 1 % of the columns 20 times larger, as hidden states have them."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return x * torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.01, 20.0, 1.0)


def _spread(s, rows, cols, block_rows):
    """The scale of every value, from one for each block."""
    s = s.repeat_interleave(BLOCK, -1)[..., :cols]
    return s if block_rows == 1 else s.repeat_interleave(block_rows, -2)[..., :rows, :]


def _weights(g, experts, n, k):
    """e4m3 weights [experts, n, k] from N(0, 0.02), with the fp32 scales of a checkpoint (the
    block's largest value over 448)."""
    q = torch.empty((experts, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((experts, _blocks(n), _blocks(k)), device="cuda")
    for e in range(experts):
        w = torch.zeros((_blocks(n) * BLOCK, _blocks(k) * BLOCK), device="cuda")
        w[:n, :k] = torch.randn((n, k), generator=g, device="cuda") * 0.02
        s[e] = w.view(_blocks(n), BLOCK, _blocks(k), BLOCK).abs().amax((1, 3)) / E4M3_MAX
        q[e] = (w[:n, :k] / _spread(s[e], n, k, BLOCK)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, s


def _quantise(x, block_rows=1):
    """x fp32 -> e4m3 and the least power of two s for each block with max|x| <= 448 s (1 for zeros)."""
    rows, cols = x.shape
    r = -(-rows // block_rows)
    p = torch.zeros((r * block_rows, _blocks(cols) * BLOCK), device=x.device)
    p[:rows, :cols] = x.abs()
    top = p.view(r, block_rows, _blocks(cols), BLOCK).amax((1, 3))
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    s = torch.where(top > 0, ((e + 127).to(torch.int32) << 23).view(torch.float32), 1.0)
    return (x / _spread(s, rows, cols, block_rows)).to(torch.float8_e4m3fn), s


def _ids(g, case):
    """Each token's experts: the top_k of logits N(0, 1) with a bias for each expert, so that the
    experts' loads differ; -1 for pairs that are dropped."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn((t, e), generator=g, device="cuda") + 0.4 * torch.randn((e,), generator=g, device="cuda")
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = ids[:, :k].to(torch.int32).contiguous()
    w = torch.softmax(top[:, :k], dim=1).contiguous()
    if case["dropped"]:
        ids[torch.rand((t, k), generator=g, device="cuda") < case["dropped"]] = -1
    return ids, w


def _sort(ids, experts):
    """row_slot [T k] (-1 past the last expert), slot_row [T, k] (-1: no expert), offsets [E + 1]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    sorted_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(sorted_key, torch.arange(experts + 1, device=ids.device))
    row = torch.arange(flat.numel(), device=ids.device)
    row_slot = torch.where(sorted_key < experts, order, -1)
    slot_row = torch.empty_like(row)
    slot_row[order] = torch.where(sorted_key < experts, row, -1)
    return row_slot.to(torch.int32), slot_row.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "product":
        rows, n, k, experts = case["rows"], case["n"], case["k"], case["experts"]
        s["a"], s["sa"] = _quantise(_activations(g, rows, k))
        s["w"], s["sw"] = _weights(g, max(1, experts), n, k)
        s["y"] = torch.empty((rows, n), dtype=DT[case["out"]], device="cuda")
        s["offsets"] = None
        if experts:
            of_row = torch.randint(0, experts, (rows,), generator=g, device="cuda")
            s["offsets"] = _sort(of_row.view(rows, 1), experts)[2]
            s["most"] = int(s["offsets"].diff().max())
        else:
            s["w"], s["sw"] = s["w"][0], s["sw"][0]
        return s
    if op == "quantise":
        s["x"] = _activations(g, case["rows"], case["k"]).to(DT[case["in"]])
        s["q"] = torch.empty((case["rows"], case["k"]), dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.empty((-(-case["rows"] // case["block_rows"]), _blocks(case["k"])), device="cuda")
        return s
    tokens, top_k, experts, h = case["tokens"], case["top_k"], case["experts"], case["h"]
    rows = tokens * top_k
    s["ids"], s["weights"] = _ids(g, case)
    s["plan"] = _sort(s["ids"], experts)
    if op == "experts":
        s["a"], s["sa"] = _quantise(_activations(g, rows, h))
        s["wg"], s["sg"] = _weights(g, experts, case["i"], h)
        s["wu"], s["su"] = _weights(g, experts, case["i"], h)
        s["wd"], s["sd"] = _weights(g, experts, h, case["i"])
        s["most"] = max(1, int(s["plan"][2].diff().max()))
        s["y"] = torch.empty((rows, h), dtype=torch.bfloat16, device="cuda")
        return s
    kind = DT[case["in"]]
    s["rows"] = torch.randn((rows, h), generator=g, device="cuda").to(kind)
    if op == "dispatch":
        s["x"] = _activations(g, tokens, h).to(kind)
        s["xs"] = torch.empty((rows, h), dtype=kind, device="cuda")
        s["y"] = torch.empty((tokens, h), device="cuda")
    else:
        s["dy"] = torch.randn((tokens, h), generator=g, device="cuda")
        s["dxs"] = torch.randn((rows, h), generator=g, device="cuda").to(kind)
        s["drows"] = torch.empty((rows, h), dtype=kind, device="cuda")
        s["dw"] = torch.empty((tokens, top_k), device="cuda")
        s["dx"] = torch.empty((tokens, h), device="cuda")
    return s


# ---- plain forms ---------------------------------------------------------------------------

def _values(q, s, block_rows=1):
    return q.float() * _spread(s, q.shape[-2], q.shape[-1], block_rows)


def _places(offsets, rows, experts, most):
    """Row -> its expert, and its place in [experts, most] (one more place for rows of no expert)."""
    row = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long(), row, right=True)
    some = e.clamp(max=experts - 1)
    return some, torch.where(e < experts, some * most + row - offsets.long()[some], experts * most), (e < experts)


def _grouped(x, w, sw, offsets, most):
    """x [rows, k] fp32 times the transposed weights of each row's expert; 0 for rows of none."""
    experts, n, k = w.shape
    rows = x.shape[0]
    e, place, some = _places(offsets, rows, experts, most)
    if rows <= experts:  # few rows: each takes its own expert's weights
        of_row = _values(w.view(torch.uint8)[e].view(torch.float8_e4m3fn), sw[e], BLOCK)
        return torch.bmm(of_row, x.view(rows, k, 1)).view(rows, n) * some[:, None]
    padded = torch.zeros((experts * most + 1, k), device=x.device)
    padded[place] = torch.where(some[:, None], x, 0.0)
    y = torch.zeros((experts * most + 1, n), device=x.device)
    y[:-1] = torch.bmm(padded[:-1].view(experts, most, k), _values(w, sw, BLOCK).transpose(1, 2)).view(-1, n)
    return y[place]


def _gathered(rows, slot_row):
    """rows of each (token, slot), fp32; 0 where there is none."""
    r = slot_row.long()
    return torch.where((r >= 0)[..., None], rows[r.clamp(min=0)].float(), 0.0)


def run(state):
    op = state["case"]["op"]
    if own:
        from quantized_ffn_gb300 import zffn
        if op == "product":
            return zffn.fp8_matmul(state["a"], state["sa"], state["w"], state["sw"], offsets=state["offsets"], y=state["y"])
        if op == "quantise":
            return zffn.fp8_quantize(state["x"], block_rows=state["case"]["block_rows"], q=state["q"], scale=state["s"])
        if op == "experts":
            return zffn.fp8_experts(state["a"], state["sa"], state["wg"], state["sg"], state["wu"], state["su"],
                                    state["wd"], state["sd"], offsets=state["plan"][2], y=state["y"])
        if op == "dispatch":
            plan = zffn.moe_sort(state["ids"], state["case"]["experts"])
            xs = zffn.moe_dispatch(state["x"], plan, out=state["xs"])
            y = zffn.moe_combine(state["rows"], plan, state["weights"], y=state["y"])
            return plan.row_slot, plan.slot_row, plan.offsets, xs, y
        plan = zffn.MoePlan(*state["plan"])
        drows, dw = zffn.moe_combine_grad(state["dy"], state["rows"], plan, state["weights"], drows=state["drows"], dweights=state["dw"])
        return drows, dw, zffn.moe_combine(state["dxs"], plan, None, y=state["dx"])
    if op == "product":
        x = _values(state["a"], state["sa"])
        if state["offsets"] is None:
            y = x @ _values(state["w"], state["sw"], BLOCK).T
        else:
            y = _grouped(x, state["w"], state["sw"], state["offsets"], state["most"])
        return y.to(state["y"].dtype)
    if op == "quantise":
        return _quantise(state["x"].float(), state["case"]["block_rows"])
    if op == "experts":
        offsets, most = state["plan"][2], state["most"]
        x = _values(state["a"], state["sa"])
        gate = _grouped(x, state["wg"], state["sg"], offsets, most)
        up = _grouped(x, state["wu"], state["su"], offsets, most)
        h = _values(*_quantise(gate / (1.0 + torch.exp(-gate)) * up))
        return _grouped(h, state["wd"], state["sd"], offsets, most).to(torch.bfloat16)
    if op == "dispatch":
        row_slot, slot_row, offsets = _sort(state["ids"], state["case"]["experts"])
        token = row_slot.long().clamp(min=0) // state["case"]["top_k"]
        xs = torch.where((row_slot >= 0)[:, None], state["x"][token], 0.0)
        y = (_gathered(state["rows"], slot_row) * state["weights"][..., None]).sum(1)
        return row_slot, slot_row, offsets, xs, y
    row_slot, slot_row, _ = state["plan"]
    slot = row_slot.long().clamp(min=0)
    drows = state["dy"][slot // state["case"]["top_k"]] * state["weights"].view(-1)[slot][:, None]
    drows = torch.where((row_slot >= 0)[:, None], drows, 0.0).to(state["rows"].dtype)
    dw = (_gathered(state["rows"], slot_row) * state["dy"][:, None, :]).sum(2)
    return drows, dw, _gathered(state["dxs"], slot_row).sum(1)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "product":
        m, n, k, e = case["rows"], case["n"], case["k"], max(1, min(case["experts"], case["rows"]))
        return {"bytes": m * k + 4 * m * _blocks(k) + e * (n * k + 4 * _blocks(n) * _blocks(k)) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    if op == "quantise":
        r = -(-case["rows"] // case["block_rows"])
        return {"bytes": case["rows"] * case["k"] * (3 if case["in"] == "bf16" else 5) + 4 * r * _blocks(case["k"]), "flops": 2 * case["rows"] * case["k"]}
    t, k, h, e = case["tokens"], case["top_k"], case["h"], case["experts"]
    p = t * k
    size = 2 if case.get("in", "bf16") == "bf16" else 4
    if op == "experts":
        i = case["i"]
        return {"bytes": p * h + 4 * p * _blocks(h) + min(e, p) * (3 * h * i + 12 * _blocks(h) * _blocks(i)) + 2 * p * h, "flops": 6 * p * h * i}
    if op == "dispatch":
        return {"bytes": 16 * p + 4 * e + t * h * size + 2 * p * h * size + 4 * t * h, "flops": 2 * p * h}
    return {"bytes": 12 * p + 4 * t * h + 3 * p * h * size + 4 * t * h, "flops": 4 * p * h}


# ---- the definitions in 64 bits ------------------------------------------------------------

def _power_of_two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(v):
    """The nearest e4m3 value (ties to the even one), of |v| <= 448: 3 bits after the first, down to steps of 2^-9."""
    _, e = torch.frexp(v)
    step = _power_of_two((e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantise(x, block_rows=1):
    rows, cols = x.shape
    q, s = torch.empty_like(x), torch.empty((-(-rows // block_rows), _blocks(cols)), dtype=torch.float64, device=x.device)
    for b in range(_blocks(cols)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        top = part.abs().amax(1)
        if block_rows > 1:
            top = torch.stack([c.amax() for c in top.split(block_rows)])
        scale = _power_of_two(torch.ceil(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** -126))))
        scale = torch.where(scale / 2 * E4M3_MAX >= top, scale / 2, scale)
        scale = torch.where(scale * E4M3_MAX < top, scale * 2, scale)
        s[:, b] = torch.where(top > 0, scale, 1.0)
        q[:, b * BLOCK:(b + 1) * BLOCK] = _exact_e4m3(part / s[:, b].repeat_interleave(block_rows)[:rows, None])
    return q, s


def _exact_values(q, s, block_rows):
    at = torch.arange(q.shape[1], device=q.device) // BLOCK
    up = torch.arange(q.shape[0], device=q.device) // block_rows
    return q.double() * s.double()[up][:, at]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return _exact_quantise(s["x"].double(), case["block_rows"])
    if op == "product":
        x = _exact_values(s["a"], s["sa"], 1)
        if s["offsets"] is None:
            return x @ _exact_values(s["w"], s["sw"], BLOCK).T
        y = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device="cuda")
        cut = s["offsets"].tolist()
        for e in range(case["experts"]):
            y[cut[e]:cut[e + 1]] = x[cut[e]:cut[e + 1]] @ _exact_values(s["w"][e], s["sw"][e], BLOCK).T
        return y
    if op == "experts":
        x = _exact_values(s["a"], s["sa"], 1)
        y = torch.zeros((x.shape[0], case["h"]), dtype=torch.float64, device="cuda")
        cut = s["plan"][2].tolist()
        for e in range(case["experts"]):
            if cut[e] == cut[e + 1]:
                continue
            xe = x[cut[e]:cut[e + 1]]
            gate = xe @ _exact_values(s["wg"][e], s["sg"][e], BLOCK).T
            up = xe @ _exact_values(s["wu"][e], s["su"][e], BLOCK).T
            h = _exact_values(*_exact_quantise(gate * torch.sigmoid(gate) * up), 1)
            y[cut[e]:cut[e + 1]] = h @ _exact_values(s["wd"][e], s["sd"][e], BLOCK).T
        return y
    t, k = case["tokens"], case["top_k"]
    _, slot_row, offsets = s["plan"]
    r = slot_row.long()
    some = (r >= 0).double()[..., None]
    if op == "dispatch":
        y = torch.zeros((t, case["h"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            y += some[:, j] * s["rows"][r[:, j].clamp(min=0)].double() * s["weights"][:, j, None].double()
        xs = torch.zeros((t * k, case["h"]), dtype=torch.float64, device="cuda")
        at = (r.view(-1) >= 0).nonzero().view(-1)
        xs[r.view(-1)[at]] = s["x"][at // k].double()
        return None, None, None, xs, y
    dy = s["dy"].double()
    drows = torch.zeros((t * k, case["h"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    dx = torch.zeros_like(dy)
    for j in range(k):
        at = (r[:, j] >= 0).nonzero().view(-1)
        rj = r[at, j]
        drows[rj] = dy[at] * s["weights"][at, j, None].double()
        dw[at, j] = (dy[at] * s["rows"][rj].double()).sum(1)
        dx[at] += s["dxs"][rj].double()
    return drows, dw, dx

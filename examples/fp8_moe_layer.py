"""A routed layer on 8-bit weights, forward and back to what feeds it, by the public entry points.

Weights are e4m3 with one fp32 scale for each 128 x 128 block, made here from fp32 matrices by
zffn.fp8_quantize.  Forward: router -> sort by expert -> rows quantised and dispatched -> the
experts' SwiGLU products -> weighted sum per token.  Backward, with the experts' weights frozen: the
gradients of the weighted sum by the experts' rows and by the routing weights (a router trains on the
latter), the gradient by the down projection's input as a product on the transposed weights, and the
dispatch's gradient by the tokens.

    python examples/fp8_moe_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_ffn_gb300 import zffn  # noqa: E402


def make_layer(E, H, I, generator):
    """Stacked (weights, scales) of the gate, up and down projections."""
    out = []
    for rows, cols in ((I, H), (I, H), (H, I)):
        q = torch.empty((E, rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((E, -(-rows // 128), -(-cols // 128)), device="cuda")
        for e in range(E):
            w = torch.randn((rows, cols), generator=generator, device="cuda") * 0.02
            zffn.fp8_quantize(w, block_rows=128, q=q[e], scale=s[e])
        out += [q, s]
    return out


def transposed(q, s):
    """The layer of the gradient by the input: a block's scale goes with its block."""
    qt = q.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
    return qt, s.transpose(1, 2).contiguous()


def forward(x, logits, top_k, layer):
    """(y fp32 [T, H], what the backward pass needs): step by step what zffn.moe_swiglu_fp8 does."""
    ids, weights = zffn.moe_router_topk(logits, top_k)
    plan = zffn.moe_sort(ids, logits.shape[1])
    xq, xs = zffn.fp8_quantize(x)
    rows_q, rows_s = zffn.moe_dispatch(xq, plan, scale=xs)
    rows = zffn.fp8_experts(rows_q, rows_s, *layer, offsets=plan.offsets)      # bf16 [T * top_k, H]
    return zffn.moe_combine(rows, plan, weights), (ids, weights, plan, rows)


def backward(dy, saved, down_t):
    """(gradient of the experts' rows, of the routing weights, of h = the down projection's input)."""
    _, weights, plan, rows = saved
    drows, dweights = zffn.moe_combine_grad(dy, rows, plan, weights)
    gq, gs = zffn.fp8_quantize(drows)
    dh = zffn.fp8_matmul(gq, gs, *down_t, offsets=plan.offsets)                # fp32 [T * top_k, I]
    return drows, dweights, dh


def main(T=256, E=16, H=1024, I=512, top_k=4, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    layer = make_layer(E, H, I, g)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    y, saved = forward(x, logits, top_k, layer)
    ids, weights, plan, rows = saved
    whole = zffn.moe_swiglu_fp8(x, ids, weights, *layer)
    dy = torch.randn((T, H), generator=g, device="cuda")
    drows, dweights, dh = backward(dy, saved, transposed(layer[4], layer[5]))
    # rows' gradients that reach the tokens themselves (as through a layer that keeps H): the dispatch's gradient
    dx = zffn.moe_combine(drows, plan)
    status = zffn.get_device_error()
    print(f"y {tuple(y.shape)} |y| {y.norm().item():.4f}, the same in one call: {torch.equal(y, whole)}, "
          f"rows an expert {plan.offsets.diff().tolist()}, |dw| {dweights.norm().item():.4f}, "
          f"|dh| {dh.norm().item():.4f}, |dx| {dx.norm().item():.4f}, device status {zffn.status_string(status)}")
    return dict(x=x, logits=logits, layer=layer, y=y, whole=whole, saved=saved, dy=dy, drows=drows, dweights=dweights, dh=dh, dx=dx)


if __name__ == "__main__":
    main()

"""A routed layer on 8-bit weights, forward and back to what feeds it, by the public entry points.

Weights are e4m3 with one fp32 scale for each 128 x 128 block, made here from fp32 matrices by
zffn.fp8_quantize.  Forward: router -> sort by expert -> rows quantised and dispatched -> the
experts' SwiGLU products -> weighted sum per token.  Backward, with the experts' weights frozen: the
gradients of the weighted sum by the experts' rows and by the routing weights (a router trains on the
latter); through the experts as products on the transposed weights, with SwiGLU's derivative between
them in torch (gate and up values are computed again); and the dispatch's gradient by the tokens.  The
quantisations of x and h pass gradients straight through, and gradients are quantised before a product.
The entry points are not known to autograd: this is the way back by hand.

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
    """(y fp32 [T, H], what the backward pass needs, the experts' 8-bit rows): step by step what
    zffn.moe_swiglu_fp8 does."""
    ids, weights = zffn.moe_router_topk(logits, top_k)
    plan = zffn.moe_sort(ids, logits.shape[1])
    xq, xs = zffn.fp8_quantize(x)
    fed = zffn.moe_dispatch(xq, plan, scale=xs)
    rows = zffn.fp8_experts(*fed, *layer, offsets=plan.offsets)                # bf16 [T * top_k, H]
    return zffn.moe_combine(rows, plan, weights), (ids, weights, plan, rows), fed


def backward(dy, saved, fed, layer, layer_t):
    """The gradients of the experts' rows, of the routing weights, of h = the down projection's input,
    and of the tokens x.  layer_t: the transposed gate, up and down projections, as layer has them."""
    _, weights, plan, rows = saved
    drows, dweights = zffn.moe_combine_grad(dy, rows, plan, weights)
    product = lambda a, w: zffn.fp8_matmul(*a, *w, offsets=plan.offsets)       # noqa: E731
    dh = product(zffn.fp8_quantize(drows), layer_t[4:6])                       # fp32 [T * top_k, I]
    gate, up = product(fed, layer[0:2]), product(fed, layer[2:4])
    s = torch.sigmoid(gate)
    dgate, dup = dh * up * s * (1 + gate * (1 - s)), dh * gate * s
    dxs = product(zffn.fp8_quantize(dgate), layer_t[0:2]) + product(zffn.fp8_quantize(dup), layer_t[2:4])
    return drows, dweights, dh, zffn.moe_combine(dxs, plan)


def main(T=256, E=16, H=1024, I=512, top_k=4, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    layer = make_layer(E, H, I, g)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    y, saved, fed = forward(x, logits, top_k, layer)
    ids, weights, plan, rows = saved
    whole = zffn.moe_swiglu_fp8(x, ids, weights, *layer)
    dy = torch.randn((T, H), generator=g, device="cuda")
    layer_t = [t for i in (0, 2, 4) for t in transposed(layer[i], layer[i + 1])]
    drows, dweights, dh, dx = backward(dy, saved, fed, layer, layer_t)
    status = zffn.get_device_error()
    print(f"y {tuple(y.shape)} |y| {y.norm().item():.4f}, the same in one call: {torch.equal(y, whole)}, "
          f"rows an expert {plan.offsets.diff().tolist()}, |dw| {dweights.norm().item():.4f}, "
          f"|dh| {dh.norm().item():.4f}, |dx| {dx.norm().item():.4f}, device status {zffn.status_string(status)}")
    return dict(x=x, logits=logits, layer=layer, y=y, whole=whole, saved=saved, fed=fed, dy=dy, drows=drows, dweights=dweights, dh=dh, dx=dx)


if __name__ == "__main__":
    main()

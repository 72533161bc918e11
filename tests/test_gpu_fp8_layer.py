"""The 8-bit routed layer's example, forward and back, against the same layer in 64 bits on its
dequantised weights.

Tolerances.  y: the experts' rows are held to a bound in test_gpu_fp8.py; here the layer as a whole:
h and the rows are rounded to e4m3 and bf16 on both sides at the same places, so y differs by e4m3
bytes that fall on the other side of a border (rare), by bf16 roundings (half a step, 2^-8 of a row's
value) and by fp32 sums: 2^-7 of the largest |y| covers them.  dweights: <dy, rows> in fp32 over H
terms against 64 bits on the same bf16 rows.  dh: the product's bound on the same quantised rows."""
import os
import sys

import pytest
import torch

from quantized_ffn_gb300 import zffn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import fp8_moe_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def values(q, s, block_rows):
    up = s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]
    if block_rows > 1:
        up = up.repeat_interleave(block_rows, -2)[..., :q.shape[-2], :]
    return q.double() * up


@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 144, 3), (64, 16, 1024, 512, 4), (600, 4, 512, 272, 2)])
def test_layer_forward_and_back(T, E, H, I, k):
    r = ex.main(T=T, E=E, H=H, I=I, top_k=k, seed=T)
    assert torch.equal(r["y"], r["whole"])
    ids, weights, plan, rows = r["saved"]
    wg, wu, wd = (values(r["layer"][2 * i], r["layer"][2 * i + 1], 128) for i in range(3))
    xv = values(*zffn.fp8_quantize(r["x"]), 1)
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            g, u = wg[e] @ xv[t], wu[e] @ xv[t]
            hq, hs = zffn.fp8_quantize((g / (1 + torch.exp(-g)) * u).float()[None])
            y[t] += weights[t, j].double() * (wd[e] @ values(hq, hs, 1)[0]).to(torch.bfloat16).double()
    assert (r["y"].double() - y).abs().max() <= 2.0 ** -7 * y.abs().max()
    # gradients
    sr = plan.slot_row.long()
    got = rows.double()[sr]
    dw, mag = (got * r["dy"].double()[:, None]).sum(2), (got * r["dy"].double()[:, None]).abs().sum(2)
    assert torch.all((r["dweights"].double() - dw).abs() <= 2 * (H / 32 + 5) * U32 * mag)
    gq, gs = zffn.fp8_quantize(r["drows"])
    gv = values(gq, gs, 1)
    for e in range(E):
        at = slice(int(plan.offsets[e]), int(plan.offsets[e + 1]))
        want, m = gv[at] @ wd[e], gv[at].abs() @ wd[e].abs()
        assert torch.all((r["dh"][at].double() - want).abs() <= (18 + 2 * (-(-H // 128))) * U32 * m + 1e-37)
    assert zffn.get_device_error() == zffn.OK


def test_no_workspace_grows_after_reserve():
    # a routed call of the reserved sizes allocates nothing
    T, E, H, I, k = 96, 8, 512, 64, 4
    zffn.release()
    zffn.reserve(T, H, I, E, k)
    held = zffn.workspace_bytes()
    ex.main(T=T, E=E, H=H, I=I, top_k=k)
    assert zffn.workspace_bytes() == held


def test_routed_call_in_a_graph():
    T, E, H, I, k = 40, 8, 256, 144, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    layer = ex.make_layer(E, H, I, g)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids, w = zffn.moe_router_topk(torch.randn((T, E), generator=g, device="cuda"), k)
    y = torch.empty((T, H), device="cuda")
    zffn.moe_swiglu_fp8(x, ids, w, *layer, y=y)          # (allocates before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zffn.moe_swiglu_fp8(x, ids, w, *layer, y=y)
    x.copy_(torch.randn((T, H), generator=g, device="cuda"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, zffn.moe_swiglu_fp8(x, ids, w, *layer))


def test_calls_back_to_back_on_one_stream():
    # programmatic launches in a chain: every call sees the one before it complete
    T, E, H, I, k = 33, 4, 256, 128, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    layer = ex.make_layer(E, H, I, g)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids, w = zffn.moe_router_topk(torch.randn((T, E), generator=g, device="cuda"), k)
    y, z = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), device="cuda")
    for _ in range(20):
        zffn.moe_swiglu_fp8(x, ids, w, *layer, y=y, accumulate=True)
    for _ in range(20):                                  # the same, each call waited for
        zffn.moe_swiglu_fp8(x, ids, w, *layer, y=z, accumulate=True)
        torch.cuda.synchronize()
    assert torch.equal(y, z) and y.abs().max() > 0
    # weights written by the kernel just before the product that reads them
    q, s = zffn.fp8_quantize(x)
    wf = torch.randn((400, H), generator=g, device="cuda")
    wq, ws = zffn.fp8_quantize(wf, block_rows=128)
    torch.cuda.synchronize()
    want = zffn.fp8_matmul(q, s, wq, ws)
    for _ in range(10):
        wq.view(torch.uint8).zero_()
        zffn.fp8_quantize(wf, block_rows=128, q=wq, scale=ws)
        assert torch.equal(zffn.fp8_matmul(q, s, wq, ws), want)


def test_routes_that_change_from_call_to_call():
    # the same memory holds another routing in every call of a chain (offsets are read before the
    # down product's wait); each result as when the call is waited for
    E, H, I, n = 16, 256, 256, 24
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    layer = ex.make_layer(E, H, I, g)
    for P in (8, 200, 4000):
        a, s = zffn.fp8_quantize(torch.randn((P, H), generator=g, device="cuda"))
        cuts = torch.sort(torch.randint(0, P + 1, (n, E + 1), generator=g, device="cuda", dtype=torch.int32), dim=1)[0]
        cuts[:, 0] = 0
        offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        chain, waited = (torch.empty((n, P, H), device="cuda") for _ in range(2))
        for i in range(n):
            zffn.fp8_experts(a, s, *layer, offsets=cuts[i].contiguous(), y=waited[i])
            torch.cuda.synchronize()
        for i in range(n):
            offsets.copy_(cuts[i])
            zffn.fp8_experts(a, s, *layer, offsets=offsets, y=chain[i])
        assert torch.equal(chain, waited)
    for T in (1, 33):
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        routes = [zffn.moe_router_topk(torch.randn((T, E), generator=g, device="cuda"), 2) for _ in range(n)]
        chain, waited = (torch.empty((n, T, H), device="cuda") for _ in range(2))
        for i in range(n):
            zffn.moe_swiglu_fp8(x, *routes[i], *layer, y=waited[i])
            torch.cuda.synchronize()
        for i in range(n):
            zffn.moe_swiglu_fp8(x, *routes[i], *layer, y=chain[i])
        assert torch.equal(chain, waited)
    assert zffn.get_device_error() == zffn.OK

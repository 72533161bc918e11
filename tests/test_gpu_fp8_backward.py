"""The way back through the 8-bit routed layer's example, from h's gradient (held to the product's bound in
test_gpu_fp8_layer.py) to the tokens', against 64 bits with SwiGLU's derivative by autograd.

Tolerance: gate and up values are products (their bound as in test_gpu_fp8.py); SwiGLU's derivative carries
their errors on (|silu'| <= 1.1, |silu''| <= 0.5, 16 fp32 roundings of a sigmoid and its products, which
grow with the gate); the two gradients are then rounded to e4m3: half a step is 2^-4 of a value, or 2^-10 of
the block's scale below its normal values, which is less than 2^-17 of the block's largest; last come the
products on the transposed weights and k fp32 sums."""
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


def largest(d):
    """The largest magnitude of each value's block of 128 columns."""
    pad = torch.nn.functional.pad(d.abs(), (0, -d.shape[1] % 128))
    return pad.view(d.shape[0], pad.shape[1] // 128, 128).amax(2).repeat_interleave(128, 1)[:, :d.shape[1]]


@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 144, 3), (64, 16, 1024, 512, 4), (600, 4, 512, 272, 2)])
def test_gradient_of_the_tokens(T, E, H, I, k):
    r = ex.main(T=T, E=E, H=H, I=I, top_k=k, seed=T + 1)
    _, _, plan, _ = r["saved"]
    wg, wu, _ = (values(r["layer"][2 * i], r["layer"][2 * i + 1], 128) for i in range(3))
    x, dh = values(*r["fed"], 1), r["dh"].double()
    c1, c2 = (18 + 2 * (-(-H // 128))) * U32, (18 + 2 * (-(-I // 128))) * U32
    want, tol = torch.zeros((T * k, H), dtype=torch.float64, device="cuda"), torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        at = slice(int(plan.offsets[e]), int(plan.offsets[e + 1]))
        g, u = (x[at] @ wg[e].T).requires_grad_(), (x[at] @ wu[e].T).requires_grad_()
        dg, du = torch.autograd.grad(torch.nn.functional.silu(g) * u, (g, u), dh[at])
        g, u, d = g.detach(), u.detach(), dh[at].abs()
        eg, eu = c1 * (x[at].abs() @ wg[e].abs().T), c1 * (x[at].abs() @ wu[e].abs().T)
        off_g = d * (1.1 * eu + 0.5 * u.abs() * eg) + 16 * U32 * d * u.abs() * (1 + g.abs())
        off_u = d * 1.1 * eg + 16 * U32 * du.abs() * (1 + g.abs())
        for v, off, w in ((dg, off_g, wg[e]), (du, off_u, wu[e])):
            step = off + 2.0 ** -4 * (v.abs() + off) + 2.0 ** -17 * largest(v.abs() + off)
            want[at] += v @ w
            tol[at] += step @ w.abs() + (c2 + U32) * ((v.abs() + step) @ w.abs())
    rows = plan.slot_row.long()
    dx, bound = want[rows].sum(1), (tol[rows] + 2 * k * U32 * (want[rows].abs() + tol[rows])).sum(1)
    assert torch.all((r["dx"].double() - dx).abs() <= bound)
    # the roundings of a row's gradients are independent of each other, so the whole is far nearer than that bound
    assert (r["dx"].double() - dx).norm() <= 2.0 ** -4 * dx.norm()
    assert zffn.get_device_error() == zffn.OK

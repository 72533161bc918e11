"""SwiGLU and its gradient against 64 bits and against differences.

Tolerance: silu(g) u takes an exponential, an addition, a division and two products in fp32.  The exponential of
x is off by a few units of 2^-24 and by |x| 2^-24 for its argument's rounding; with 8 (1 + |g|) 2^-24 of the
value for the forward pass, and 16 (1 + |g|) 2^-24 of each term's magnitude for the gradient
(1 - s is as exact as s, absolutely, where s is near 1: |g| (1 - s) is then below 1).  A bf16 result adds half a step."""
import math

import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu


def forms(gu, dh):
    I = gu.shape[1] // 2
    g, u, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    s = torch.sigmoid(g)
    grow = (1 + g.abs()) * ref.U32
    h = g * s * u
    dg, du = d * u * s * (1 + g * torch.sigmoid(-g)), d * g * s
    dg_tol = 16 * grow * (d * u * s).abs() * (1 + g.abs() * torch.sigmoid(-g)) + 4 * ref.U32 * (d * u * s * g).abs()
    return (h, 8 * grow * h.abs()), (torch.cat((dg, du), 1), torch.cat((dg_tol, 16 * grow * du.abs()), 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,I", [(1, 1), (1, 8), (3, 7), (5, 130), (37, 768), (64, 1021), (300, 2052), (1, 65537), (40000, 24)])
def test_forward_and_gradient(rows, I, dtype):
    gen = ref.generator(rows + I)
    gu, dh = ref.randn(gen, rows, 2 * I, scale=3.0, dtype=dtype), ref.randn(gen, rows, I, dtype=dtype)
    (h, h_tol), (dgu, d_tol) = forms(gu, dh)
    ref.check(zffn.swiglu(gu), h, h_tol, dtype)
    ref.check(zffn.swiglu_grad(dh, gu), dgu, d_tol, dtype)
    out = torch.full((rows, I), 9.0, dtype=dtype, device="cuda")
    assert zffn.swiglu(gu, h=out) is out
    inplace = gu.clone()
    assert torch.equal(zffn.swiglu_grad(dh, inplace, dgu=inplace), zffn.swiglu_grad(dh, gu))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_rows(dtype):
    gen = ref.generator(5)
    for off in (1, 2, 3, 4):
        flat = ref.randn(gen, off + 9 * 64, dtype=dtype)
        gu, dh = flat[off:].view(9, 64), ref.randn(gen, off + 9 * 32, dtype=dtype)[off:].view(9, 32)
        (h, h_tol), (dgu, d_tol) = forms(gu, dh)
        ref.check(zffn.swiglu(gu), h, h_tol, dtype)
        ref.check(zffn.swiglu_grad(dh, gu), dgu, d_tol, dtype)


def test_special_values():
    inf, nan = math.inf, math.nan
    g = torch.tensor([[0.0, -0.0, 100.0, -100.0, 1e30, -1e30, inf, -inf, nan, 1.0, -3e38, 88.0, -88.0, -104.0]], device="cuda")
    u = torch.full_like(g, 2.0)
    gu = torch.cat((g, u), 1)
    h = zffn.swiglu(gu)[0].cpu()
    assert h[0] == 0 and h[1] == 0 and h[2] == 200 and abs(h[3]) < 1e-36 and h[4] == 2e30 and h[5] == 0 and h[6] == inf
    assert math.isnan(h[7]) and math.isnan(h[8]) and h[10] == 0 and h[11] == 176 and abs(h[12]) < 1e-35 and abs(h[13]) < 1e-36
    d = zffn.swiglu_grad(torch.ones_like(g), gu)[0].cpu()
    n = g.shape[1]
    assert d[0] == 1 and d[2] == 2 and d[4] == 2 and d[5] == 0 and d[n + 4] == 1e30 and d[n + 5] == 0 and d[n] == 0
    assert torch.isfinite(d[[0, 1, 2, 3, 4, 5, 9, 10, 11, 12, 13]]).all() and torch.isfinite(d[[n + i for i in (0, 1, 2, 3, 4, 5, 9, 10, 11)]]).all()


def test_gradient_is_the_difference_quotient():
    # in fp32, steps of 2^-6: the quotient's own error is a sixth of the step's square times the third derivative
    # (below 1 for both, with |g|, |u| <= 2), and 2^-24 |h| / 2^-6 twice for the rounding of h
    gen = ref.generator(6)
    gu = (torch.rand((50, 64), generator=gen, device="cuda") * 4 - 2)
    dh, e = torch.randn((50, 32), generator=gen, device="cuda"), 2.0 ** -6
    d = zffn.swiglu_grad(dh, gu)
    for c in range(0, 64, 5):
        up, down = gu.clone(), gu.clone()
        up[:, c] += e
        down[:, c] -= e
        q = (zffn.swiglu(up).double() - zffn.swiglu(down).double()) / (up[:, c] - down[:, c]).double()[:, None] * dh.double()
        bound = dh.abs()[:, c % 32].double() * (e * e / 6 * 4 + 2 * 8 * 3 * ref.U32 * 8 / e)
        assert torch.all((q[:, c % 32] - d[:, c].double()).abs() <= bound)

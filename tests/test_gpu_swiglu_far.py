"""SwiGLU and its gradient of gates far below zero, where 1 / (1 + e^-g) leaves fp32's range and its product with a
large u or gradient does not, against 64 bits.

Tolerance as in test_gpu_swiglu.py, 16 (1 + |g|) 2^-24 of the value (an exponential to 2^-22, to the fourth power, is
off by 16 2^-24); 1e-37 is added for what is below fp32's normal numbers, and a bf16 result is rounded once more."""
import itertools
import math

import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu

G = [-200.0, -181.0, -170.0, -150.0, -104.0, -100.0, -90.0, -89.0, -88.0, -87.0, -80.0, -60.0, -40.0, -33.0, -32.5, -32.0, -31.5, -20.0, -3.0, 0.5, 30.0]
U = [3e38, 1e30, -1e25, 2.0, -1e-20]
D = [1e38, -1e30, 1.0, 1e-25]


def values(dtype, drop):
    """gu [1, 2 I] and dh [1, I] of all triples whose results are in range, mixed, and without the last `drop`."""
    rows = []
    for g, u, d in itertools.product(G, U, D):
        s = 1 / (1 + math.exp(-g))
        if max(abs(v) for v in (u * g * s, d * u * s * (1 + g * (1 - s)), d * g * s)) < 3e38:
            rows.append((g, u, d))
    rows += [(1.0, 1.0, 1.0)] * (-len(rows) % 8)
    t = torch.tensor(rows, dtype=torch.float64)
    t = t[torch.randperm(len(rows), generator=torch.Generator().manual_seed(3))][:len(rows) - drop]
    g, u, d = (c.to(dtype).cuda() for c in t.unbind(1))
    return torch.cat((g, u)).view(1, -1), d.view(1, -1).contiguous()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("drop", [0, 2, 4, 5])     # (packs of 16 bytes, of fewer, single values)
def test_far_gates(dtype, drop):
    gu, dh = values(dtype, drop)
    I = dh.shape[1]
    g, u, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    s, rest = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    h, dgu = u * g * s, torch.cat((d * u * s * (1 + g * rest), d * g * s), 1)
    grow = 16 * (1 + g.abs()) * ref.U32
    got = zffn.swiglu(gu)
    ref.check(got, h, grow * h.abs(), dtype)
    both = zffn.swiglu_grad(dh, gu)
    # (near the zero of 1 + g (1 - s), at g = -1.28, alone the terms' magnitudes count: no such gate is here)
    ref.check(both, dgu, torch.cat((grow, grow), 1) * dgu.abs(), dtype)
    same = gu.clone()
    assert torch.equal(zffn.swiglu_grad(dh, same, dgu=same), both)
    far = (g < -87) & (h.abs() > 1e-30)
    assert far.any() and torch.all(got[far] != 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_far_gate_leaves_its_neighbours(dtype):
    gen = ref.generator(4)
    gu, dh = ref.randn(gen, 64, 2 * 256, scale=3.0, dtype=dtype), ref.randn(gen, 64, 256, dtype=dtype)
    h, d = zffn.swiglu(gu), zffn.swiglu_grad(dh, gu)
    some = torch.rand((64, 256), generator=gen, device="cuda") < 0.1
    cold = gu.clone()
    cold[:, :256][some] = -90.0
    h2, d2 = zffn.swiglu(cold), zffn.swiglu_grad(dh, cold)
    assert torch.equal(h2[~some], h[~some])
    keep = torch.cat((~some, ~some), 1)
    assert torch.equal(d2[keep], d[keep])


def test_infinite_gates():
    inf = math.inf
    gu = torch.tensor([[-inf, -inf, -3e38, -1e5, -inf, 1.0, -3e38, -50.0, 2.0, 1e30, 3e38, 3e38, 0.0, 1.0, 0.0, inf]], device="cuda")
    h = zffn.swiglu(gu)[0].cpu()
    # silu(-inf) is NaN by the formula; silu(-3e38) and silu(-1e5) are 0 whatever finite u is
    assert h[0].isnan() and h[1].isnan() and h[4].isnan() and h[2] == 0 and h[3] == 0 and h[6] == 0 and h[7] == -inf
    d = zffn.swiglu_grad(torch.ones((1, 8), device="cuda"), gu)[0].cpu()
    assert d[0].isnan() and d[8].isnan() and d[2] == 0 and d[3] == 0 and d[10] == 0 and d[11] == 0

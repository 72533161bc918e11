"""Infinite weights and tokens of adapters: what they enter is infinite or NaN, the rest is as without them."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,r", [(9, 16), (9, 24), (700, 24)])
def test_infinite_weights(T, r):
    L, N, K = 3, 264, 136
    gen = ref.generator(T + r)
    ids = torch.randint(0, L, (T,), generator=gen, device="cuda").int()
    plan = zffn.moe_sort(ids.view(T, 1), L)
    x, dy, A, B = ref.randn(gen, T, K), ref.randn(gen, T, N), ref.randn(gen, L, r, K), ref.randn(gen, L, N, r)
    x[:, :8], A[:, :, :8], dy[:, :8], B[:, :8] = 1.0, 1.0, 1.0, 1.0
    out, v = zffn.lora_add(x, A, B, plan, dtype=torch.float32)
    grads = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    one = ids == 1
    # a weight of B: one column of out, for the adapter's tokens
    Bi = B.clone()
    Bi[1, 5, 3] = float("inf")
    got, gv = zffn.lora_add(x, A, Bi, plan, dtype=torch.float32)
    assert torch.equal(gv, v) and not torch.isfinite(got[one, 5]).any()
    got[one, 5] = out[one, 5]
    assert torch.equal(got, out)
    # a weight of A on the way back: one column of dx
    Ai = A.clone()
    Ai[1, 3, 7] = float("inf")
    dx, dA, dB = zffn.lora_grad(dy, x, v, Ai, B, plan, dtype=torch.float32)
    assert not torch.isfinite(dx[one, 7]).any()
    dx[one, 7] = grads[0][one, 7]
    assert all(torch.equal(g, w) for g, w in zip((dx, dA, dB), grads))
    # a token: one column of its adapter's dA
    xi = x.clone()
    xi[int(one.nonzero()[0]), 7] = float("inf")
    dx, dA, dB = zffn.lora_grad(dy, xi, v, A, B, plan, dtype=torch.float32)
    assert not torch.isfinite(dA[1, :, 7]).any()
    dA[1, :, 7] = grads[1][1, :, 7]
    assert all(torch.equal(g, w) for g, w in zip((dx, dA, dB), grads))

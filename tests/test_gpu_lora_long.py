"""Adapters of long projections for so many tokens that one block sums a whole row: v and dv, which are fp32, are not
to get less exact with the number of tokens.

Tolerance of positive sums: an add of 16 products to a sum of 24 bits that cuts instead of rounding loses half a last
place on the average over many adds, 2^-24 of the sum by then at most, which is half of a part's on the average (a
margin of 1.25 for values that are not even); the parts, of 512 products as the bf16 products have them, are joined with a rounding each."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref
from tests.test_gpu_bf16_long_sums import positive

pytestmark = pytest.mark.gpu

PART = 512


def bound(terms):
    return (1.25 * (min(PART, terms) / 16) / 2 + -(-terms // PART) / 2 + 2) * ref.U32


def plan_of(gen, T, L, packed):
    ids = torch.randint(0, L, (T,), generator=gen, device="cuda").int()
    return zffn.moe_sort((ids.sort()[0] if packed else ids).view(T, 1).contiguous(), L)


# (one block a row tile; 65536: several turns, 8264: not whole turns, with a cut stage; 3000 tokens: four blocks)
CASES = [(10000, 65536, 128, 1), (20000, 65536, 64, 2), (10000, 11008, 72, 1), (10000, 8264, 128, 3), (20000, 8264, 40, 1), (20000, 16456, 16, 1),
         (3000, 65536, 128, 2), (300, 65536, 128, 1)]


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("T,C,r,L", CASES)
def test_long_rows(T, C, r, L, packed):
    gen = ref.generator(T + C + r)
    plan = plan_of(gen, T, L, packed)
    x, W = positive(gen, T, C), positive(gen, L, r, C)
    scale = torch.tensor([0.5, 2.0, 1.0], device="cuda")[:L]
    want = torch.zeros((T, r), dtype=torch.float64, device="cuda")
    for e, lo, hi in ref.groups(plan.offsets, T):
        t = plan.row_slot[lo:hi].long()
        want[lo:hi] = (x[t].double() @ W[e].double().T) * float(scale[e])
    # forward: W as A
    B = positive(gen, L, 8, r)
    out, v = zffn.lora_add(x, W, B, plan, scale=scale, dtype=torch.float32)
    ref.check(v, want, bound(C) * want)
    wout = torch.zeros((T, 8), dtype=torch.float64, device="cuda")
    # back: W as B, x as dy; dx = dv A
    x8, A, Wt = positive(gen, T, 8), positive(gen, L, r, 8), W.transpose(1, 2).contiguous()
    dx, dA, dB = zffn.lora_grad(x, x8, v, A, Wt, plan, scale=scale, dtype=torch.float32)
    wdx, wdA = torch.zeros_like(wout), torch.zeros(A.shape, dtype=torch.float64, device="cuda")
    for e, lo, hi in ref.groups(plan.offsets, T):
        t = plan.row_slot[lo:hi].long()
        wout[t], wdx[t], wdA[e] = want[lo:hi] @ B[e].double().T, want[lo:hi] @ A[e].double(), want[lo:hi].T @ x8[t].double()
    ref.check(out, wout, (bound(C) + ref.sum_bound(3 * r)) * wout)
    ref.check(dx, wdx, (bound(C) + ref.sum_bound(3 * r)) * wdx)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("T,C,r", [(10000, 16392, 128), (20000, 33000, 48)])
def test_signed_rows_repeat_and_stay_apart(T, C, r):
    # turns of the accumulators leave nothing of one row in another: each row by itself, whatever the others are
    gen = ref.generator(T + r)
    plan = plan_of(gen, T, 1, False)
    x, A, B = ref.randn(gen, T, C), ref.randn(gen, 1, r, C, scale=0.05), ref.randn(gen, 1, 8, r)
    out, v = zffn.lora_add(x, A, B, plan, dtype=torch.float32)
    t = plan.row_slot[:T].long()
    want, mag = torch.empty((T, r), dtype=torch.float64, device="cuda"), torch.empty((T, r), dtype=torch.float64, device="cuda")
    for lo in range(0, T, 2000):
        rows, w = x[t[lo:lo + 2000]].double(), A[0].double().T
        want[lo:lo + 2000], mag[lo:lo + 2000] = rows @ w, rows.abs() @ w.abs()
    ref.check(v, want, bound(C) * mag)
    x[t[5]] = float("nan")
    other, w = zffn.lora_add(x, A, B, plan, dtype=torch.float32)
    assert torch.equal(w[:5], v[:5]) and torch.equal(w[6:], v[6:]) and torch.isnan(w[5]).all()
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("T,r,L", [(4096, 32, 1), (4100, 16, 2), (5000, 72, 1), (3000, 80, 1), (2500, 128, 1), (30000, 64, 3), (30000, 104, 1)])
def test_weights_gradients_of_many_tokens(T, r, L, packed):
    # dB's sums are over tokens alone, in parts of 512 of them (each in three pieces of v, whose sums meet in two
    # more roundings); dA's have dv's own error before them
    N, K = 136, 72
    gen = ref.generator(T + r)
    plan = plan_of(gen, T, L, packed)
    x, dy, A, B = positive(gen, T, K), positive(gen, T, N), positive(gen, L, r, K), positive(gen, L, N, r)
    v = torch.rand((T, r), generator=gen, device="cuda") + 0.5
    dx, dA, dB = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    rows = int(plan.offsets.diff().max())
    (_, _), (wA, _), (wB, _) = ref.lora_grad(dy, x, v, A, B, plan, None, None)
    ref.check(dB, wB, (bound(rows) + 2 * ref.U32) * wB)
    ref.check(dA, wA, (bound(rows) + bound(N) + 2 * ref.U32) * wA)
    again = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dA, dB)))
    assert zffn.get_device_error() == zffn.OK

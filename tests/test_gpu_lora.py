"""Low-rank adapters of many requests and their gradients, against 64-bit forms (tests/bf16_ref.py, which derives
the tolerances)."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def adapter_ids(gen, T, L, kind):
    ids = torch.randint(0, L, (T,), generator=gen, device="cuda").int()
    if kind == "one":
        ids[:] = L // 2
    elif kind == "none":
        ids[:] = -1
    elif kind == "mixed":
        ids[torch.rand((T,), generator=gen, device="cuda") < 0.3] = -1
        ids[torch.rand((T,), generator=gen, device="cuda") < 0.1] = L
    elif kind == "packed":
        ids = torch.sort(ids)[0]
    return ids


def inputs(T, N, K, r, L, kind):
    gen = ref.generator(T + N + K + r + L)
    ids = adapter_ids(gen, T, L, kind)
    plan = zffn.moe_sort(ids.view(T, 1), L)
    x, dy = ref.randn(gen, T, K), ref.randn(gen, T, N, scale=0.1)
    A, B = ref.randn(gen, L, r, K, scale=0.05), ref.randn(gen, L, N, r, scale=0.05)
    scale = torch.rand((L,), generator=gen, device="cuda") + 0.5
    return gen, ids, plan, x, dy, A, B, scale


SIZES = [(1, 8, 8, 8, 1), (1, 1032, 2048, 16, 8), (2, 264, 136, 8, 3), (7, 520, 264, 16, 64), (61, 2056, 1032, 16, 48), (64, 256, 4096, 64, 5),
         (130, 136, 264, 24, 2), (333, 1032, 520, 40, 5), (500, 264, 72, 128, 3), (1000, 392, 1000, 32, 4096), (2100, 520, 264, 64, 4)]
KINDS = ["random", "one", "none", "mixed", "packed"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,N,K,r,L", SIZES)
def test_forward(T, N, K, r, L, kind):
    gen, ids, plan, x, _, A, B, scale = inputs(T, N, K, r, L, kind)
    for dtype in DTYPES:
        base = ref.randn(gen, T, N, dtype=dtype)
        want, tol, wv, vtol = ref.lora(x, A, B, plan, scale, base)
        out, v = torch.full_like(base, 7.0), torch.full((T, r), 7.0, device="cuda")
        o, got_v = zffn.lora_add(x, A, B, plan, scale=scale, base=base, out=out, v=v)
        assert o is out and got_v is v
        ref.check(v, wv, vtol)
        assert torch.all(v[int(plan.offsets[L]):] == 0)
        ref.check(out, want, tol, dtype)
        rest = (ids < 0) | (ids >= L)
        assert torch.equal(out[rest], base[rest])
        same = base.clone()                                       # in place
        zffn.lora_add(x, A, B, plan, scale=scale, base=same, out=same)
        assert torch.equal(same, out)
        alone, _ = zffn.lora_add(x, A, B, plan, dtype=dtype)      # without a base and scales
        want, tol, _, _ = ref.lora(x, A, B, plan, None, None)
        assert alone.dtype == dtype
        ref.check(alone, want, tol, dtype)
        assert torch.all(alone[rest] == 0)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,N,K,r,L", SIZES)
def test_gradients(T, N, K, r, L, kind):
    gen, ids, plan, x, dy, A, B, scale = inputs(T, N, K, r, L, kind)
    _, v = zffn.lora_add(x, A, B, plan, scale=scale)
    for dtype in DTYPES:
        base = ref.randn(gen, T, K, dtype=dtype)
        dx, dA, dB = (torch.full_like(t, 7.0, dtype=dtype) for t in (x, A, B))
        got = zffn.lora_grad(dy, x, v, A, B, plan, scale=scale, base=base, dx=dx, dA=dA, dB=dB)
        assert got[0] is dx and got[1] is dA and got[2] is dB
        for g, (want, tol) in zip(got, ref.lora_grad(dy, x, v, A, B, plan, scale, base)):
            ref.check(g, want, tol, dtype)
        same = base.clone()
        zffn.lora_grad(dy, x, v, A, B, plan, scale=scale, base=same, dx=same)
        assert torch.equal(same, dx)
        alone = zffn.lora_grad(dy, x, v, A, B, plan, dtype=dtype)
        for g, (want, tol) in zip(alone, ref.lora_grad(dy, x, v, A, B, plan, None, None)):
            assert g.dtype == dtype
            ref.check(g, want, tol, dtype)
    assert zffn.get_device_error() == zffn.OK


def test_gradients_are_differences():
    # out is linear in A, in B and in x, so a difference of any step is the gradient; fp32 results, steps of 1:
    # the two forward sums' own tolerances, and a bf16 input that is a whole number plus the step is exact
    gen = ref.generator(9)
    T, N, K, r, L = 40, 72, 136, 16, 3
    plan = zffn.moe_sort(torch.randint(-1, L, (T, 1), generator=gen, device="cuda").int(), L)
    whole = lambda *s: torch.randint(-4, 5, s, generator=gen, device="cuda").to(torch.bfloat16)      # noqa: E731
    x, A, B, dy = whole(T, K), whole(L, r, K), whole(L, N, r), whole(T, N)
    f = lambda x, A, B: float((zffn.lora_add(x, A, B, plan, dtype=torch.float32)[0].double() * dy.double()).sum())   # noqa: E731
    _, v = zffn.lora_add(x, A, B, plan)
    grads = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    for i, t in enumerate((x, A, B)):
        for at in torch.randint(0, t.numel(), (12,), generator=gen, device="cuda").tolist():
            hi, lo = [x, A, B], [x, A, B]
            hi[i], lo[i] = t.clone(), t.clone()
            hi[i].view(-1)[at] += 1
            lo[i].view(-1)[at] -= 1
            assert (f(*hi) - f(*lo)) / 2 == float(grads[i].reshape(-1)[at])     # (whole numbers below 2^24: exact)


@pytest.mark.parametrize("T,L", [(40, 4), (700, 3)])
def test_infinities_stay_in_their_rows(T, L):
    gen, ids, plan, x, dy, A, B, scale = inputs(T, 264, 136, 16, L, "mixed")
    clean, cv = zffn.lora_add(x, A, B, plan, scale=scale)
    grads = zffn.lora_grad(dy, x, cv, A, B, plan, scale=scale)
    rest = (ids < 0) | (ids >= L)
    one = int((ids == 1).nonzero()[0])
    x[rest], dy[rest] = float("nan"), float("inf")
    x[one, 3] = float("inf")
    out, v = zffn.lora_add(x, A, B, plan, scale=scale)
    others = torch.arange(T, device="cuda") != one
    assert torch.equal(out[others], clean[others]) and not torch.isfinite(out[one]).any()
    row = int(plan.slot_row[one])
    assert torch.isinf(v[row]).all()
    got = zffn.lora_grad(dy, x, cv, A, B, plan, scale=scale)
    assert torch.equal(got[0], grads[0]) and torch.equal(got[2], grads[2])
    assert torch.equal(got[1][[0]], grads[1][[0]]) and not torch.isfinite(got[1][1][:, 3]).any()


def test_rows_that_name_no_token():
    gen, ids, plan, x, dy, A, B, scale = inputs(50, 72, 64, 8, 3, "random")
    bad = zffn.MoePlan(plan.row_slot.clone(), plan.slot_row.clone(), plan.offsets)
    for row, value in ((4, 50), (20, -1), (33, 1 << 30)):
        bad.slot_row[bad.row_slot[row].long()] = -1
        bad.row_slot[row] = value
    gone = bad.slot_row.view(-1) < 0
    out, v = zffn.lora_add(x, A, B, plan, scale=scale)
    got, gv = zffn.lora_add(x, A, B, bad, scale=scale)
    assert torch.equal(got[~gone], out[~gone]) and torch.all(got[gone] == 0) and torch.all(gv[[4, 20, 33]] == 0)
    dx, dA, dB = zffn.lora_grad(dy, x, v, A, B, bad, scale=scale)
    assert torch.all(dx[gone] == 0) and torch.isfinite(dA).all() and torch.isfinite(dB).all()
    assert zffn.get_device_error() == zffn.OK

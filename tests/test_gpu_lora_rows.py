"""Adapters of few tokens, row by row, of ranks that are no power of two (two columns a thread), against the 64-bit
forms of bf16_ref.py, which derives the tolerances; and adapters on a given stream."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref
from tests.test_gpu_lora import DTYPES, KINDS, inputs

pytestmark = pytest.mark.gpu

# ranks of less than four loads of 16 bytes, of just four and of more; columns of one block, of several and a part of one
SIZES = [(1, 8, 8, 24, 1), (5, 264, 136, 24, 6), (3, 520, 72, 56, 2), (9, 520, 264, 40, 64), (8, 264, 264, 96, 9), (3, 1032, 72, 120, 3), (40, 1032, 264, 56, 64)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,N,K,r,L", SIZES)
def test_forward_by_rows(T, N, K, r, L, kind):
    assert r & (r - 1) and zffn.load().zffn_lora_work_bytes(T, r, L, 0) == 0
    gen, ids, plan, x, _, A, B, scale = inputs(T, N, K, r, L, kind)
    rest = (ids < 0) | (ids >= L)
    for dtype in DTYPES:
        base = ref.randn(gen, T, N, dtype=dtype)
        want, tol, wv, vtol = ref.lora(x, A, B, plan, scale, base)
        out, v = torch.full_like(base, 7.0), torch.full((T, r), 7.0, device="cuda")
        zffn.lora_add(x, A, B, plan, scale=scale, base=base, out=out, v=v)
        ref.check(v, wv, vtol)
        assert torch.all(v[int(plan.offsets[L]):] == 0)
        ref.check(out, want, tol, dtype)
        assert torch.equal(out[rest], base[rest])
        same = base.clone()
        zffn.lora_add(x, A, B, plan, scale=scale, base=same, out=same)
        assert torch.equal(same, out)
        alone, _ = zffn.lora_add(x, A, B, plan, dtype=dtype)
        want, tol, _, _ = ref.lora(x, A, B, plan, None, None)
        ref.check(alone, want, tol, dtype)
        assert torch.all(alone[rest] == 0)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("T,r", [(5, 24), (7, 16), (700, 40)])
def test_results_on_a_given_stream(T, r):
    # the inputs are made, and the results read, on the given stream alone; v, the gradients and what the calls work
    # in come from its memory, while the current stream is kept busy and takes and gives back blocks of the same size
    N, K, L = 264, 520, 4
    _, _, plan, x, dy, A, B, scale = inputs(T, N, K, r, L, "mixed")
    want = zffn.lora_add(x, A, B, plan, scale=scale)
    want = (*want, *zffn.lora_grad(dy, x, want[1], A, B, plan, scale=scale, dtype=torch.float32))
    side, load = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(4):
            load = load @ load * 1e-2
        with torch.cuda.stream(side):
            x2, dy2 = x.clone(), dy.clone()
        out, v = zffn.lora_add(x2, A, B, plan, scale=scale, stream=side)
        grads = zffn.lora_grad(dy2, x2, v, A, B, plan, scale=scale, dtype=torch.float32, stream=side)
        for n in (v.numel() * 4, 2 * T * 2 * 128, 2 * T * 2 * 64):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        with torch.cuda.stream(side):
            same = [torch.equal(g, w) for g, w in zip((out, v, *grads), want)]
        assert all(same), same
    torch.cuda.synchronize()
    assert zffn.get_device_error() == zffn.OK

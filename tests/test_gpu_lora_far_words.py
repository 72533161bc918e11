"""Rows of adapters that name no token, by words as far out as there are: a sum with one of them does not pass for a token."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu

MOST, LEAST = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("T,r", [(60, 16), (60, 24), (900, 16), (900, 72)])
@pytest.mark.parametrize("words", [[MOST], [LEAST], [MOST, LEAST], [MOST - 1, MOST], [MOST - 1, MOST, LEAST, LEAST + 1]])
def test_words_that_are_no_token(T, r, words):
    L, N, K, gone = 3, 264, 136, len(words)
    gen = ref.generator(T + r)
    # adapter 1 has these rows alone
    ids = torch.randint(0, 2, (T,), generator=gen, device="cuda").int() * 2
    ids[10:10 + gone] = 1
    plan = zffn.moe_sort(ids.view(T, 1), L)
    x, dy, A, B = ref.randn(gen, T, K), ref.randn(gen, T, N), ref.randn(gen, L, r, K), ref.randn(gen, L, N, r)
    out, v = zffn.lora_add(x, A, B, plan, dtype=torch.float32)
    grads = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    lo = int(plan.offsets[1])
    bad = zffn.MoePlan(plan.row_slot.clone(), plan.slot_row.clone(), plan.offsets)
    bad.row_slot[lo:lo + gone] = torch.tensor(words, dtype=torch.int32, device="cuda")
    bad.slot_row[10:10 + gone] = -1
    got, gv = zffn.lora_add(x, A, B, bad, dtype=torch.float32)
    back = zffn.lora_grad(dy, x, v, A, B, bad, dtype=torch.float32)
    keep = ids != 1
    assert torch.equal(got[keep], out[keep]) and torch.all(got[~keep] == 0) and torch.all(gv[lo:lo + gone] == 0)
    assert torch.equal(back[0][keep], grads[0][keep]) and torch.all(back[0][~keep] == 0)
    for g, w in zip(back[1:], grads[1:]):
        assert torch.equal(g[[0, 2]], w[[0, 2]]) and torch.all(g[1] == 0)
    assert zffn.get_device_error() == zffn.OK

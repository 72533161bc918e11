"""Long sums of the bf16 products and adapters.  The tensor core's adds may cut off what is below the accumulator's
last bit, so that a long sum of positive values comes out short; the kernels sum in parts, joined in fp32."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu


def part_bound(part, terms):
    """Of positive bf16 products: a part adds 16 at a time and may lose 4 * 2^-24 of what it has by then, half its
    sum on the average (a margin of 1.25 for values that are not even); a join rounds what there is by then."""
    return (1.25 * 4 * (min(part, terms) / 16) / 2 + -(-terms // part) / 2 + 2) * ref.U32


def positive(gen, *shape):
    return (torch.rand(shape, generator=gen, device="cuda") + 0.5).bfloat16()


# (one token and a few: K over clusters; 65 rows of 24 experts and many tiles of 300 rows: small tiles, large ones, pairs)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,N,K,E", [(1, 136, 65536, 0), (300, 264, 65536, 0), (260, 1032, 8200, 24), (1560, 1032, 8200, 24),
                                     (4800, 520, 8200, 24), (3000, 1032, 2056, 0)])
def test_products_of_positive_values(M, N, K, E, transposed):
    gen = ref.generator(M + N + K)
    a, w = positive(gen, M, K), positive(gen, max(E, 1), K, N) if transposed else positive(gen, max(E, 1), N, K)
    offsets = ref.cuts(M, E, "even") if E else None
    y = zffn.bf16_matmul(a, w if E else w[0], offsets, transposed, dtype=torch.float32)
    want, _ = ref.product(a, w if E else w[0], offsets, transposed)
    ref.check(y, want, part_bound(512, K) * want)
    yb = zffn.bf16_matmul(a, w if E else w[0], offsets, transposed)
    ref.check(yb, want, part_bound(K, K) * want, torch.bfloat16)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("M,N,K,E", [(3000, 136, 264, 0), (70000, 136, 64, 0), (70000, 72, 136, 300), (20000, 2056, 1032, 20), (300001, 136, 16, 0)])
def test_weights_gradients_of_positive_values(M, N, K, E):
    gen = ref.generator(M + N + K)
    dy, a = positive(gen, M, N), positive(gen, M, K)
    # (300 groups: nearly all rows are one's)
    offsets = None if not E else ref.cuts(M, E, "even") if E < 100 else ref.cuts(M, E, "one")
    rows = M if E != 20 else M // E
    dw = zffn.bf16_matmul_grad_w(dy, a, offsets, dtype=torch.float32)
    want = ref.grad_w(dy, a, offsets)[0].view(dw.shape)
    ref.check(dw, want, part_bound(512, rows) * want)
    dwb = zffn.bf16_matmul_grad_w(dy, a, offsets)
    ref.check(dwb, want, part_bound(4096 if M > 1 << 18 else rows, rows) * want, torch.bfloat16)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("r", [16, 64, 72, 80, 128])
def test_adapters_of_many_tokens(r, packed):
    T, N, K, L = 21000, 136, 1096, 2
    gen = ref.generator(r + packed)
    ids = (torch.rand((T,), generator=gen, device="cuda") < 0.3).int()
    if packed:
        ids = torch.sort(ids)[0]
    plan = zffn.moe_sort(ids.view(T, 1), L)
    x, dy, A, B = positive(gen, T, K), positive(gen, T, N), positive(gen, L, r, K), positive(gen, L, N, r)
    out, v = zffn.lora_add(x, A, B, plan, dtype=torch.float32)
    dx, dA, dB = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    want, tol, wv, vtol = ref.lora(x, A, B, plan, None, None)
    ref.check(v, wv, vtol)
    ref.check(out, want, tol)
    wanted = ref.lora_grad(dy, x, v, A, B, plan, None, None)
    ref.check(dx, *wanted[0])
    # dv's own error (of N values, and the same sums in parts of 512 at least), then the tokens' in parts of 4096
    few = int((ids == 1).sum())
    for g, (w, _), e in ((dA, wanted[1], part_bound(512, N)), (dB, wanted[2], 0.0)):
        ref.check(g, w, (e + part_bound(4096, T - few) + 2 * ref.U32) * w.abs())
    again = zffn.lora_grad(dy, x, v, A, B, plan, dtype=torch.float32)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dA, dB)))
    assert zffn.get_device_error() == zffn.OK

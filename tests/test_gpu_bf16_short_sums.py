"""Sums whose result is bf16: it is the nearest bf16 value of an fp32 sum, or of one that close to it, since what the
tensor core's adds cut off a long sum would now and then move it to the next.

Tolerance: half a step at the value itself, and the bound of test_gpu_lora_long.py on sums of positive products in
parts of 512."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref
from tests.test_gpu_bf16_long_sums import positive
from tests.test_gpu_lora_long import bound

pytestmark = pytest.mark.gpu


def nearest(got, want, tol):
    step = torch.exp2(torch.floor(torch.log2(want)) - 7)
    off = (got.double() - want).abs() - step / 2
    assert torch.all(off <= tol), (int((off > tol).sum()), off.max(), tol.max())


# (small tiles, with K over clusters and without; large ones, single and in pairs)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,N,K,E", [(1, 4104, 65536, 0), (8, 2056, 2048, 8), (300, 1032, 2048, 24), (2000, 2056, 2048, 24), (3000, 1032, 4096, 0),
                                     (3000, 1032, 16384, 0), (3000, 1032, 65536, 0), (2000, 264, 32768, 3), (6000, 1032, 2056, 24)])
def test_products(M, N, K, E, transposed):
    gen = ref.generator(M + N + K)
    a, w = positive(gen, M, K), positive(gen, max(E, 1), K, N) if transposed else positive(gen, max(E, 1), N, K)
    offsets = ref.cuts(M, E, "even") if E else None
    y = zffn.bf16_matmul(a, w if E else w[0], offsets, transposed)
    want, _ = ref.product(a, w if E else w[0], offsets, transposed)
    nearest(y, want, bound(K) * want)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("M,N,K,E", [(2048, 1032, 520, 0), (4096, 2056, 1032, 0), (65536, 520, 264, 0), (262144, 136, 72, 0), (16000, 1032, 520, 20), (70000, 136, 264, 9)])
def test_weights_gradients(M, N, K, E):
    gen = ref.generator(M + N + K)
    dy, a = positive(gen, M, N), positive(gen, M, K)
    offsets = ref.cuts(M, E, "one" if E == 9 else "even") if E else None
    dw = zffn.bf16_matmul_grad_w(dy, a, offsets)
    want = ref.grad_w(dy, a, offsets)[0].view(dw.shape)
    some = want > 0
    nearest(dw[some], want[some], bound(M if E != 20 else M // E) * want[some])
    assert torch.all(dw[~some] == 0)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("T,r", [(4096, 16), (5000, 64), (30000, 40)])
def test_adapters_weights_gradients(T, r):
    N, K = 1032, 264
    gen = ref.generator(T + r)
    plan = zffn.moe_sort(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1)
    x, dy, A, B = positive(gen, T, K), positive(gen, T, N), positive(gen, 1, r, K), positive(gen, 1, N, r)
    v = torch.rand((T, r), generator=gen, device="cuda") + 0.5
    _, dA, dB = zffn.lora_grad(dy, x, v, A, B, plan)
    (_, _), (wA, _), (wB, _) = ref.lora_grad(dy, x, v, A, B, plan, None, None)
    # (two roundings more for the sums of v's three pieces; dA: dv's own error first)
    nearest(dB, wB, (bound(T) + 2 * ref.U32) * wB)
    nearest(dA, wA, (bound(T) + bound(N) + 2 * ref.U32) * wA)
    assert zffn.get_device_error() == zffn.OK

"""Long sums whose result is bf16: they are rounded by half a step at most, which what the tensor core's adds cut off
is not to be seen beside.  Sums near a power of two, where a bf16 step is the largest part of the value.

Tolerance: half a step, and the positive sums' bound of test_gpu_lora_long.py for parts of 4096 products."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref
from tests.test_gpu_bf16_long_sums import positive

pytestmark = pytest.mark.gpu


def bound(part, terms):
    return (1.25 * (min(part, terms) / 16) / 2 + -(-terms // part) / 2 + 2) * ref.U32


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,N,K,E", [(3000, 1032, 16384, 0), (3000, 1032, 65536, 0), (2000, 264, 32768, 3), (1, 136, 65536, 0), (300, 264, 65536, 0)])
def test_products(M, N, K, E, transposed):
    gen = ref.generator(M + N + K)
    a, w = positive(gen, M, K), positive(gen, max(E, 1), K, N) if transposed else positive(gen, max(E, 1), N, K)
    offsets = ref.cuts(M, E, "even") if E else None
    y = zffn.bf16_matmul(a, w if E else w[0], offsets, transposed)
    want, _ = ref.product(a, w if E else w[0], offsets, transposed)
    ref.check(y, want, bound(4096, K) * want, torch.bfloat16)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("M,N,K,E", [(65536, 520, 264, 0), (131072, 136, 72, 0), (262144, 136, 72, 0), (70000, 136, 264, 9)])
def test_weights_gradients(M, N, K, E):
    gen = ref.generator(M + N + K)
    dy, a = positive(gen, M, N), positive(gen, M, K)
    offsets = ref.cuts(M, E, "one") if E else None
    dw = zffn.bf16_matmul_grad_w(dy, a, offsets)
    want = ref.grad_w(dy, a, offsets)[0].view(dw.shape)
    ref.check(dw, want, bound(4096, M) * want, torch.bfloat16)
    assert zffn.get_device_error() == zffn.OK

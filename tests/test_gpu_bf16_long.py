"""Weights' gradients that take more than a second, the bound of a single wait: the warp that zeroes the rows past an
expert's last has none to zero until the last expert's tiles, and its wait may not be counted from the kernel's begin.
145 GB of operands and results; corners of the gradients in 64 bits."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_no_wait_lasts_as_long_as_the_gradients():
    M, N, K = 2 ** 20, 32768, 32768
    gen = ref.generator(1)
    dy, a = (torch.empty((M, n), dtype=torch.bfloat16, device="cuda") for n in (N, K))
    for t in (dy, a):
        for i in range(0, M, 2 ** 16):
            t[i:i + 2 ** 16].normal_(generator=gen)
    cut = torch.tensor([0, M - 16, M - 8], dtype=torch.int32, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    dw = zffn.bf16_matmul_grad_w(dy, a, cut)
    end.record()
    torch.cuda.synchronize()
    assert zffn.get_device_error() == zffn.OK
    assert begin.elapsed_time(end) > 1000
    for n, k in ((0, 0), (N - 64, K - 64), (N // 2, 256)):
        for e, lo, hi in ((0, 0, M - 16), (1, M - 16, M - 8)):
            d, x = dy[lo:hi, n:n + 64].double(), a[lo:hi, k:k + 64].double()
            ref.check(dw[e, n:n + 64, k:k + 64], d.T @ x, ref.sum_bound(hi - lo) * (d.abs().T @ x.abs()), torch.bfloat16)

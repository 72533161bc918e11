"""A product of CTA pairs that takes seconds (229376 x 262144 x 65536: more than 4e9 clocks, the bound of
a single wait): no role's bounded wait may begin with the kernel and last as long as it does.  152 GB of
operands and result; a corner of the result in 64 bits, with the products' tolerance."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests.test_gpu_fp8 import check_product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_no_wait_lasts_as_long_as_the_product():
    M, N, K = 229376, 262144, 65536
    gen = torch.Generator(device="cuda").manual_seed(1)

    def operand(rows, block_rows):      # (not negative, no NaN)
        q = torch.randint(0, 0x7F, (rows, K), dtype=torch.uint8, device="cuda", generator=gen)
        s = torch.rand((-(-rows // block_rows), K // 128), device="cuda", generator=gen) + 0.5
        return q, s

    a, sa = operand(M, 1)
    w, sw = operand(N, 128)
    y = zffn.fp8_matmul(a, sa, w, sw, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert zffn.get_device_error() == zffn.OK
    for r, c in ((0, 0), (M - 2, N - 128), (130000, 131072)):
        x = zffn.fp8_dequant(a[r:r + 2], sa[r:r + 2]).double()
        v = zffn.fp8_dequant(w[c:c + 128], sw[c // 128:c // 128 + 1], block_rows=128).double()
        want = (x @ v.T).cpu().numpy()
        # (the operands' values are rounded to fp32 above: 2^-24 each)
        check_product(y[r:r + 2, c:c + 128], want, want * (1 + 2.0 ** -23), K, torch.bfloat16)

"""Results made for a given stream belong to that stream's memory: a block that the current stream has
just let go of, with its own kernels still writing there, is not taken for them."""
import pytest
import torch

from quantized_ffn_gb300 import zffn

pytestmark = pytest.mark.gpu


def busy_then_free(like):
    """The current stream writes sevens for some milliseconds into memory that is free afterwards."""
    block = torch.empty_like(like)
    for _ in range(300):
        block.fill_(7)
    del block


@pytest.mark.parametrize("which", ["product", "quantise", "combine"])
def test_results_on_a_given_stream(which):
    T, K = 4096, 4096
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, K), generator=gen, device="cuda")
    q, s = zffn.fp8_quantize(x)
    w, ws = zffn.fp8_quantize(torch.randn((K, K), generator=gen, device="cuda"), block_rows=128)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    plan = zffn.moe_sort(ids, 1)
    run = {"product": lambda **kw: zffn.fp8_matmul(q, s, w, ws, **kw),
           "quantise": lambda **kw: zffn.fp8_quantize(x, **kw)[0],
           "combine": lambda **kw: zffn.moe_combine(x, plan, None, **kw)}[which]
    want = run()
    like = torch.empty_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy_then_free(like)
    got = run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert zffn.get_device_error() == zffn.OK

"""A stream of another device is refused by the 8-bit and sorting functions before anything is made or
launched (its handle would be taken for one of the current device)."""
import types

import pytest
import torch

from quantized_ffn_gb300 import zffn

pytestmark = pytest.mark.gpu


def test_stream_of_another_device_is_refused():
    here = torch.cuda.current_device()
    other = types.SimpleNamespace(cuda_stream=0, device_index=here + 1)     # (a stand-in: there is one device)
    same = types.SimpleNamespace(cuda_stream=0)                             # (a bare handle is the current device's)
    x = torch.ones((4, 256), device="cuda")
    q, s = zffn.fp8_quantize(x, stream=same)
    w, ws = zffn.fp8_quantize(torch.ones((128, 256), device="cuda"), block_rows=128)
    ids = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    plan = zffn.moe_sort(ids, 1, stream=same)
    one = torch.ones((4, 1), device="cuda")
    for call in (lambda **kw: zffn.fp8_quantize(x, **kw), lambda **kw: zffn.fp8_dequant(q, s, **kw),
                 lambda **kw: zffn.fp8_matmul(q, s, w, ws, **kw), lambda **kw: zffn.moe_sort(ids, 1, **kw),
                 lambda **kw: zffn.moe_dispatch(x, plan, **kw), lambda **kw: zffn.moe_combine(x, plan, **kw),
                 lambda **kw: zffn.moe_combine_grad(x, x, plan, one, **kw)):
        with pytest.raises(ValueError, match="stream must be on the current device"):
            call(stream=other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = zffn.fp8_quantize(x, stream=side)
    side.synchronize()
    assert torch.equal(got.view(torch.uint8), q.view(torch.uint8))

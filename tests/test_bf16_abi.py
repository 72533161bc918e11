"""Refusals of the bf16 products, SwiGLU and the adapters, on the host: bad arguments are rejected before the
device is touched."""
import ctypes

import pytest
import torch

from quantized_ffn_gb300 import build as zbuild
from quantized_ffn_gb300 import zffn

F = ctypes.c_void_p(0x10000)      # never dereferenced: the checks reject first
ODD = ctypes.c_void_p(0x10001)
A2, A4, A8 = (ctypes.c_void_p(0x10000 + i) for i in (2, 4, 8))
BAD = zffn.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    return zffn.load()


@pytest.mark.parametrize("bad", [dict(a=None), dict(w=None), dict(y=None), dict(off=None), dict(dt=2), dict(dt=-1), dict(M=0), dict(M=(1 << 24) + 1),
                                 dict(N=0), dict(N=65537), dict(K=0), dict(K=100), dict(K=65544), dict(E=0), dict(E=4097), dict(t=1, N=100),
                                 dict(a=A8), dict(w=A8), dict(off=A2), dict(y=A2), dict(dt=1, y=ODD)])
def test_product_refuses(lib, bad):
    v = {**dict(a=F, w=F, off=F, t=0, dt=0, y=F, M=4, N=104, K=256, E=3), **bad}
    assert lib.zffn_bf16_matmul(*(v[k] for k in ("a", "w", "off", "t", "dt", "y", "M", "N", "K", "E")), None) == BAD


@pytest.mark.parametrize("bad", [dict(dy=None), dict(a=None), dict(dw=None), dict(off=None), dict(dt=2), dict(M=0), dict(N=100), dict(N=0), dict(K=12),
                                 dict(E=0), dict(E=4097), dict(dy=A8), dict(a=A8), dict(dw=A8), dict(off=A2), dict(M=(1 << 24) + 1)])
def test_weights_gradient_refuses(lib, bad):
    v = {**dict(dy=F, a=F, off=F, dt=0, dw=F, M=4, N=104, K=256, E=3), **bad}
    assert lib.zffn_bf16_matmul_grad_w(*(v[k] for k in ("dy", "a", "off", "dt", "dw", "M", "N", "K", "E")), None) == BAD


@pytest.mark.parametrize("args", [(2, F, F, 4, 8), (0, None, F, 4, 8), (0, F, None, 4, 8), (0, F, F, 0, 8), (0, F, F, 4, 0), (0, F, F, 1 << 31, 8),
                                  (0, F, F, 4, (1 << 20) + 1), (0, A2, F, 4, 8), (0, F, A2, 4, 8), (1, ODD, F, 4, 8), (1, F, ODD, 4, 8)])
def test_swiglu_refuses(lib, args):
    dt, gu, h, rows, i = args
    assert lib.zffn_swiglu(dt, gu, h, rows, i, None) == BAD
    assert lib.zffn_swiglu_grad(dt, F, gu, h, rows, i, None) == BAD
    if gu is not F:
        assert lib.zffn_swiglu_grad(dt, gu, F, F, rows, i, None) == BAD


LORA = dict(dy=F, x=F, v=F, A=F, B=F, s=F, rs=F, sr=F, off=F, dt=0, base=F, out=F, wdt=0, dA=F, dB=F, dv=F, work=F, T=4000, N=64, K=256, r=16, L=3)
SHARED = ([{k: None} for k in ("x", "A", "B", "rs", "sr", "off", "out", "v", "work")] +
          [dict(dt=2), dict(T=0), dict(T=(1 << 24) + 1), dict(N=60), dict(N=0), dict(N=65544), dict(K=4), dict(K=65544), dict(r=0), dict(r=12),
           dict(r=136), dict(L=0), dict(L=4097), dict(x=A8), dict(A=A8), dict(B=A8), dict(base=A8), dict(out=A8), dict(v=A8), dict(work=A8), dict(s=A2), dict(rs=A2),
           dict(sr=A2), dict(off=A2)])


@pytest.mark.parametrize("bad", SHARED)
def test_adapters_refuse(lib, bad):
    v = {**LORA, **bad}
    assert lib.zffn_lora_add(*(v[k] for k in ("x", "A", "B", "s", "rs", "sr", "off", "dt", "base", "out", "v", "work", "T", "N", "K", "r", "L")), None) == BAD


@pytest.mark.parametrize("bad", SHARED + [{k: None} for k in ("dy", "dA", "dB", "dv")] + [dict(wdt=3), dict(dy=A8), dict(dA=A8), dict(dB=A8), dict(dv=A8)])
def test_adapters_gradients_refuse(lib, bad):
    v = {**LORA, **bad}
    keys = ("dy", "x", "v", "A", "B", "s", "rs", "sr", "off", "dt", "base", "out", "wdt", "dA", "dB", "dv", "work", "T", "N", "K", "r", "L")
    assert lib.zffn_lora_grad(*(v[k] for k in keys), None) == BAD


def test_work_bytes(lib):
    assert lib.zffn_lora_work_bytes(4000, 24, 3, 0) == 4000 * 2 * 128 and lib.zffn_lora_work_bytes(400, 24, 3, 1) == 2 * 400 * 2 * 128
    assert lib.zffn_lora_work_bytes(1, 16, 8, 0) == 0 and lib.zffn_lora_work_bytes(1, 16, 8, 1) == 2 * 2 * 64      # (row by row)
    assert all(lib.zffn_lora_work_bytes(*bad, 1) == 0 for bad in ((0, 16, 1), (4, 12, 1), (4, 136, 1), (1 << 25, 16, 1), (4, 16, 0), (4, 16, 4097)))


def test_reason_is_given(lib):
    assert lib.zffn_bf16_matmul(F, F, None, 1, 0, F, 4, 100, 256, 1, None) == BAD
    assert b"N must be a multiple of 8" in lib.zffn_last_error()
    assert lib.zffn_lora_add(F, F, F, None, F, F, F, 0, None, F, F, F, 4, 64, 256, 20, 1, None) == BAD
    assert b"r must be a multiple of 8" in lib.zffn_last_error()


def test_python_checks():
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)                   # noqa: E731
    plan = zffn.MoePlan(torch.zeros(4).int(), torch.zeros((4, 1)).int(), torch.zeros(3).int())
    two = zffn.MoePlan(torch.zeros(4).int(), torch.zeros((2, 2)).int(), torch.zeros(3).int())
    x, A, B = b(4, 64), b(2, 8, 64), b(2, 16, 8)
    for bad in (lambda: zffn.bf16_matmul(b(4, 64), b(8, 32)), lambda: zffn.bf16_matmul(b(4, 64), b(64, 8), transposed=False),
                lambda: zffn.bf16_matmul(b(4, 64), b(2, 8, 64)), lambda: zffn.bf16_matmul(b(4, 64).float(), b(8, 64)),
                lambda: zffn.bf16_matmul(b(4, 64), b(8, 64)),                                        # not on the GPU
                lambda: zffn.bf16_matmul(b(4, 64), b(2, 8, 64), offsets=torch.zeros(2).int()),
                lambda: zffn.bf16_matmul_grad_w(b(4, 8), b(3, 64)), lambda: zffn.bf16_matmul_grad_w(b(4, 8), b(4, 64), offsets=torch.zeros(()).int()),
                lambda: zffn.bf16_matmul_grad_w(b(4, 8), b(4, 64), offsets=torch.zeros(0).int()),
                lambda: zffn.swiglu(b(4, 7)), lambda: zffn.swiglu(b(4, 8).half()), lambda: zffn.swiglu(b(8)), lambda: zffn.swiglu(b(4, 8)),
                lambda: zffn.swiglu_grad(b(4, 3), b(4, 8)), lambda: zffn.swiglu_grad(b(4, 4).float(), b(4, 8)),
                lambda: zffn.lora_add(x, A, B, plan), lambda: zffn.lora_add(x, A, b(2, 16, 16), plan), lambda: zffn.lora_add(x, b(2, 8, 32), B, plan),
                lambda: zffn.lora_add(b(2, 64), A, B, two), lambda: zffn.lora_add(x, A, B, plan[:2]),
                lambda: zffn.lora_grad(b(4, 8), x, torch.zeros((4, 8)), A, B, plan)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        zffn._native().swiglu(x)

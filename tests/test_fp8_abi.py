"""Refusals of the block-scaled 8-bit entry points and of the sort by expert, on the host: bad
arguments are rejected before the device is touched; and the plain reference forms on known values."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import build as zbuild
from quantized_ffn_gb300 import zffn
from tests import f8_ref as ref

F = ctypes.c_void_p(0x10000)      # never dereferenced: the checks reject first
ODD = ctypes.c_void_p(0x10001)
A4 = ctypes.c_void_p(0x10004)
BAD = zffn.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    return zffn.load()


@pytest.mark.parametrize("args", [(2, F, F, F, 4, 128, 1), (0, None, F, F, 4, 128, 1), (0, F, None, F, 4, 128, 1),
                                  (0, F, F, None, 4, 128, 1), (0, F, F, F, 0, 128, 1), (0, F, F, F, 4, 0, 1),
                                  (0, F, F, F, 4, 128, 64), (0, F, F, F, 1 << 31, 128, 1), (0, F, F, F, 1, (1 << 20) + 1, 1),
                                  (0, ctypes.c_void_p(0x10002), F, F, 4, 128, 1), (1, ODD, F, F, 4, 128, 1), (0, F, F, ODD, 4, 128, 1)])
def test_quantize_refuses(lib, args):
    assert lib.zffn_fp8_quantize(*args, None) == BAD
    if args[0] == 0:
        d, x, q, s, r, c, b = args
        if x is None or not isinstance(x, ctypes.c_void_p) or x.value == F.value:
            assert lib.zffn_fp8_dequant(q, s, x, r, c, b, None) == BAD


GOOD = dict(a=F, sa=F, w=F, sw=F, off=F, dt=0, y=F, M=4, N=100, K=256, E=3)


@pytest.mark.parametrize("bad", [dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(dt=2), dict(dt=-1),
                                 dict(M=0), dict(M=(1 << 24) + 1), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=100),
                                 dict(K=65552), dict(E=0), dict(E=4097), dict(off=None), dict(a=A4), dict(w=A4), dict(sa=ODD),
                                 dict(sw=ODD), dict(off=ODD), dict(y=ODD), dict(dt=1, y=ODD), dict(N=1 << 20, E=4096)])
def test_matmul_refuses(lib, bad):
    v = {**GOOD, **bad}
    assert lib.zffn_fp8_matmul(v["a"], v["sa"], v["w"], v["sw"], v["off"], v["dt"], v["y"], v["M"], v["N"], v["K"], v["E"], None) == BAD


EXP = dict(a=F, sa=F, off=F, wg=F, sg=F, wu=F, su=F, wd=F, sd=F, dt=1, y=F, P=4, H=256, I=128, E=3)


@pytest.mark.parametrize("bad", [{k: None} for k in ("a", "sa", "wg", "sg", "wu", "su", "wd", "sd", "y", "off")] +
                         [dict(dt=5), dict(P=0), dict(H=0), dict(H=250), dict(I=8), dict(I=100), dict(E=0), dict(E=5000),
                          dict(wg=A4), dict(wu=A4), dict(wd=A4), dict(a=A4), dict(sg=ODD), dict(y=ODD)])
def test_experts_refuse(lib, bad):
    v = {**EXP, **bad}
    assert lib.zffn_fp8_experts(*(v[k] for k in ("a", "sa", "off", "wg", "sg", "wu", "su", "wd", "sd", "dt", "y", "P", "H", "I", "E")), None) == BAD


@pytest.mark.parametrize("bad", [{k: None} for k in ("x", "ids", "w", "wg", "sg", "wu", "su", "wd", "sd", "y")] +
                         [dict(T=0), dict(H=100), dict(I=0), dict(E=0), dict(k=0), dict(k=65), dict(T=1 << 24, k=2), dict(x=ODD), dict(y=ODD),
                          dict(wg=A4)])
def test_routed_block_refuses(lib, bad):
    v = {**dict(x=F, ids=F, w=F, wg=F, sg=F, wu=F, su=F, wd=F, sd=F, y=F, T=4, H=256, I=128, E=8, k=2), **bad}
    assert lib.zffn_moe_swiglu_fp8(*(v[n] for n in ("x", "ids", "w", "wg", "sg", "wu", "su", "wd", "sd", "y", "T", "H", "I", "E", "k")), 0, None) == BAD


@pytest.mark.parametrize("args", [(None, F, F, F, 4, 8, 2), (F, None, F, F, 4, 8, 2), (F, F, None, F, 4, 8, 2), (F, F, F, None, 4, 8, 2),
                                  (F, F, F, F, 0, 8, 2), (F, F, F, F, 4, 0, 2), (F, F, F, F, 4, 4097, 2), (F, F, F, F, 4, 8, 0),
                                  (F, F, F, F, 4, 8, 65), (F, F, F, F, 1 << 24, 8, 2), (ODD, F, F, F, 4, 8, 2), (F, F, F, ODD, 4, 8, 2)])
def test_sort_refuses(lib, args):
    assert lib.zffn_moe_sort(*args, None) == BAD


@pytest.mark.parametrize("args", [(None, 64, None, 0, F, F, F, None, 4, 2), (F, 0, None, 0, F, F, F, None, 4, 2),
                                  (F, (1 << 20) + 1, None, 0, F, F, F, None, 4, 2), (F, 64, F, 0, F, F, F, None, 4, 2),
                                  (F, 64, None, 2, F, F, F, None, 4, 2), (F, 64, F, 2, F, F, F, None, 4, 2), (F, 64, None, -1, F, F, F, None, 4, 2),
                                  (F, 64, None, 0, None, F, F, None, 4, 2), (F, 64, None, 0, F, None, F, None, 4, 2),
                                  (F, 64, None, 0, F, F, None, None, 4, 2), (F, 64, None, 0, F, F, F, None, 0, 2),
                                  (F, 64, None, 0, ODD, F, F, None, 4, 2), (F, 64, ODD, 2, F, F, F, F, 4, 2)])
def test_dispatch_refuses(lib, args):
    assert lib.zffn_moe_dispatch(*args, None) == BAD


@pytest.mark.parametrize("args", [(3, F, F, F, F, 4, 64, 2, 0), (0, None, F, F, F, 4, 64, 2, 0), (0, F, None, F, F, 4, 64, 2, 0),
                                  (0, F, F, F, None, 4, 64, 2, 0), (0, F, F, F, F, 0, 64, 2, 0), (0, F, F, F, F, 4, 0, 2, 0),
                                  (0, F, F, F, F, 4, 65537, 2, 0), (0, F, F, F, F, 4, 64, 65, 0), (0, ODD, F, F, F, 4, 64, 2, 0),
                                  (1, ODD, F, F, F, 4, 64, 2, 0), (0, F, F, ODD, F, 4, 64, 2, 0), (0, F, F, F, ODD, 4, 64, 2, 0)])
def test_combine_refuses(lib, args):
    assert lib.zffn_moe_combine(*args, None) == BAD


@pytest.mark.parametrize("args", [(0, None, F, F, F, F, F, F, 4, 64, 2), (0, F, None, F, F, F, F, F, 4, 64, 2), (0, F, F, None, F, F, F, F, 4, 64, 2),
                                  (0, F, F, F, None, F, F, F, 4, 64, 2), (0, F, F, F, F, None, F, F, 4, 64, 2), (0, F, F, F, F, F, None, None, 4, 64, 2),
                                  (7, F, F, F, F, F, F, F, 4, 64, 2), (0, F, F, F, F, F, F, F, 4, 0, 2), (1, F, F, F, F, F, ODD, F, 4, 64, 2)])
def test_combine_grad_refuses(lib, args):
    assert lib.zffn_moe_combine_grad(*args, None) == BAD


def test_reason_is_given(lib):
    assert lib.zffn_fp8_matmul(F, F, F, F, None, 0, F, 4, 100, 100, 1, None) == BAD
    assert b"K must be a multiple of 16" in lib.zffn_last_error()


def test_python_checks_shapes():
    f = torch.float8_e4m3fn
    a, sa = torch.zeros((4, 256)).to(f), torch.zeros((4, 2))
    with pytest.raises(ValueError):
        zffn.fp8_matmul(a, sa, torch.zeros((8, 128)).to(f), torch.zeros((1, 2)))      # K differs
    with pytest.raises(ValueError):
        zffn.fp8_quantize(torch.zeros((4, 256)), block_rows=32)
    with pytest.raises(ValueError):
        zffn.fp8_quantize(torch.zeros((4, 256), dtype=torch.float16))
    with pytest.raises(ValueError):
        zffn.moe_combine(torch.zeros((3, 8)), zffn.MoePlan(torch.zeros(4).int(), torch.zeros((2, 2)).int(), torch.zeros(3).int()))
    with pytest.raises(ValueError):
        zffn.moe_sort(torch.zeros((2, 2), dtype=torch.int32), 4)                      # not on the GPU


def test_binding_checks_its_arguments():
    plan = zffn.MoePlan(torch.zeros(4).int(), torch.zeros((2, 2)).int(), torch.zeros(3).int())
    rows = torch.zeros((4, 8))
    for bad in (lambda: zffn.fp8_quantize([1.0, 2.0]), lambda: zffn.fp8_quantize(torch.zeros(8)),
                lambda: zffn.moe_combine(rows, (plan[0], plan[1])), lambda: zffn.moe_combine(rows, plan, accumulate=True),
                lambda: zffn.moe_combine(rows.double(), plan), lambda: zffn.moe_dispatch(torch.zeros((3, 8)), plan),
                lambda: zffn.moe_combine_grad(torch.zeros((2, 7)), rows, plan, torch.zeros((2, 2))),
                lambda: zffn.fp8_matmul(torch.zeros((4, 256)).to(torch.float8_e4m3fn), torch.zeros((4, 2)),
                                        torch.zeros((8, 256)).to(torch.float8_e4m3fn), torch.zeros((1, 2)), dtype="float32"),
                lambda: zffn.fp8_matmul(torch.zeros((4, 256)), torch.zeros((4, 2)), torch.zeros((8, 256)), torch.zeros((1, 2))),
                lambda: zffn.moe_sort(torch.zeros((2, 2), dtype=torch.int64), 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        zffn._native().moe_sort(plan[1])


# ---- the reference forms ---------------------------------------------------------------------

def test_reference_byte_values_are_torch_float8():
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.VALUES, want, equal_nan=True)
    assert ref.VALUES[0x7E] == 448 and ref.VALUES[1] == 2.0 ** -9 and np.isnan(ref.VALUES[0xFF])


def test_reference_rounding_is_nearest_even():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.01, [17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -0.0]])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.to_byte(v.astype(np.float64)), want)


def test_reference_scale_is_the_least_power_of_two():
    x = np.zeros((3, 128))
    x[0, 5], x[1, 0], x[2, 127] = 448.0, -448.5, 1e-30
    q, s = ref.quantize(x)
    assert list(s[:, 0]) == [1.0, 2.0, 2.0 ** -108]
    assert np.all(np.abs(x) <= 448 * s) and np.all(np.abs(x).max(1) > 224 * s[:, 0])


def test_reference_sort():
    row_slot, slot_row, offsets = ref.sort(np.array([[2, 0], [0, -1], [2, 9]]), 3)
    assert list(row_slot) == [1, 2, 0, 4, -1, -1] and list(offsets) == [0, 2, 2, 4]
    assert slot_row.tolist() == [[2, 0], [1, -1], [3, -1]]

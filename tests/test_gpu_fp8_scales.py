"""8-bit products whose scales' product leaves the normal fp32 numbers or comes near the largest, on small
tiles (16 and 32 rows), single large tiles and CTA pairs."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import f8_ref as ref
from tests.test_gpu_fp8 import U32, check_product, f8, f32, product_inputs

pytestmark = pytest.mark.gpu

# (rows, outputs, K)
SHAPES = [(5, 300, 272), (30, 257, 272), (300, 9728, 144), (200, 9999, 272)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_whose_product_is_subnormal(M, N, K, dtype):
    # a scales' product below 2^-126 is held in steps of 2^-149: half a step times a block's largest sum,
    # 128 * 448^2 < 2^25, for each block; a bf16 result of such size rounds in steps of 2^-133
    rng = np.random.default_rng(M + N)
    a, sa, w, sw = product_inputs(rng, M, N, K)
    sa = (2.0 ** rng.integers(-126, -118, sa.shape)).astype(np.float32)
    sw = np.exp(rng.uniform(np.log(1e-9), np.log(1e-3), sw.shape)).astype(np.float32)
    y = zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw), dtype=dtype)
    want, mag = ref.matmul(a, sa, w, sw)
    got = y.double().cpu().numpy()
    tol = (16 + 2 + 2 * ref.blocks(K)) * U32 * mag + ref.blocks(K) * 2.0 ** -125
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -134
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_whose_product_is_near_the_largest(M, N, K):
    # products of scales up to just below 2^128 times sums of 2^-18 and up: finite results, zeros stay zero
    rng = np.random.default_rng(M * N)
    a, w = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
    a[:, ::16] = rng.choice([0x01, 0x02, 0x03, 0x81], (M, len(range(0, K, 16))))      # +- 2^-9 .. 3 * 2^-9
    w[:, ::16] = rng.choice([0x00, 0x01, 0x08, 0x82], (N, len(range(0, K, 16))))
    a[::3], w[::5] = 0, 0
    sa = np.full((M, ref.blocks(K)), 2.0 ** 120, np.float32)
    sw = rng.uniform(128.0, 255.99, (ref.blocks(N), ref.blocks(K))).astype(np.float32)
    y = zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw))
    want, mag = ref.matmul(a, sa, w, sw)
    check_product(y, want, mag, K, torch.float32)
    assert torch.all(y[::3] == 0) and torch.all(y[:, ::5] == 0) and torch.all(torch.isfinite(y)) and bool((y != 0).any())

"""Offsets that no sort writes (descending, negative, past the last row, arbitrary): each entry counts as
the largest of those up to it, kept within [0, M], so that such a call ends with the results of the
ascending array that this makes, on every kind of tile."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests.gpu_util import dev
from tests.test_gpu_fp8 import expert_inputs, f8, f32, product_inputs

pytestmark = pytest.mark.gpu


def arrays(rng, M, E):
    up = np.sort(rng.integers(0, M + 1, E + 1))
    swapped = up.copy()
    swapped[[1, E]] = swapped[[E, 1]]
    low, high = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    yield np.tile([0, M], E + 1)[:E + 1]                     # every other expert claims every row
    yield np.full(E + 1, M)
    yield up[::-1]
    yield swapped
    yield rng.integers(-M, 2 * M + 1, E + 1)
    yield rng.integers(low, high, E + 1)
    yield np.tile([high, low], E + 1)[:E + 1]


# small tiles, K split over a cluster and not; more experts than a block has threads; large tiles, single and pairs
@pytest.mark.parametrize("M,N,K,E", [(8, 256, 1040, 128), (8, 16, 512, 4096), (200, 136, 2064, 5), (3000, 392, 272, 300),
                                     (1500, 5136, 272, 4), (4500, 2568, 144, 3)])
def test_product(M, N, K, E):
    rng = np.random.default_rng(M + N)
    a, sa, w, sw = product_inputs(rng, M, N, K, E)
    t = (f8(a), f32(sa), f8(w), f32(sw))
    for cut in arrays(rng, M, E):
        cut = cut.astype(np.int32)
        up = np.maximum.accumulate(np.clip(cut, 0, M))
        got, want = (torch.full((M, N), 5.0, device="cuda") for _ in range(2))
        zffn.fp8_matmul(*t, offsets=dev(cut), y=got)
        zffn.fp8_matmul(*t, offsets=dev(up), y=want)
        assert torch.equal(got, want)
        assert torch.all(got[:up[0]] == 5.0) and torch.all(got[up[E]:] == 0)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("P,H,I,E", [(8, 512, 192, 128), (300, 256, 272, 5), (1500, 144, 2576, 4)])
def test_experts(P, H, I, E):
    rng = np.random.default_rng(P + I)
    a, sa, wg, sg, wu, su, wd, sd = expert_inputs(rng, P, H, I, E)
    t = (f8(a), f32(sa), f8(wg), f32(sg), f8(wu), f32(su), f8(wd), f32(sd))
    for cut in arrays(rng, P, E):
        cut = cut.astype(np.int32)
        up = np.maximum.accumulate(np.clip(cut, 0, P))
        got, want = (torch.full((P, H), 5.0, device="cuda") for _ in range(2))
        zffn.fp8_experts(*t, offsets=dev(cut), y=got)
        zffn.fp8_experts(*t, offsets=dev(up), y=want)
        assert torch.equal(got, want)
    assert zffn.get_device_error() == zffn.OK

"""Grouped products and experts on the large tiles: single ones (more than 64 rows an expert on average)
and CTA pairs (1024 and more), with experts' borders inside tiles, experts without rows, rows of no
expert, and results whose rows are 16-byte multiples (written by TMA) and not.  Tolerances as in
test_gpu_fp8.py; of the experts, the rows at every border and some between."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests.gpu_util import dev
from tests.test_gpu_fp8 import HALF_BF16, check_product, expert_inputs, experts_ref, f8, f32, product_inputs
from tests import f8_ref as ref

pytestmark = pytest.mark.gpu


def cuts(M, E, kind):
    """Offsets: "borders" at odd places within tiles, "empty": experts without rows between and at both ends,
    "unused": rows of no expert from the middle of a tile on, "few": one expert with one row."""
    even = np.linspace(0, M, E + 1)
    if kind == "borders":
        cut = even + np.array([0] + [(37, -61, 5)[i % 3] for i in range(E - 1)] + [0])
    elif kind == "empty":
        cut = np.zeros(E + 1)
        cut[E // 2 + 1:] = M
        if E > 3:
            cut[E // 2] = M // 3
    elif kind == "unused":
        cut = even * 0.7
    else:
        cut = even.copy()
        cut[1] = 1
    return cut.astype(np.int32)


KINDS = ["borders", "empty", "unused", "few"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K,E", [(1500, 5136, 272, 4), (1500, 5137, 144, 4), (4500, 2568, 272, 3), (4500, 2570, 144, 3), (6000, 1290, 16, 60)])
def test_product(M, N, K, E, kind, dtype):
    rng = np.random.default_rng(M + N + len(kind))
    a, sa, w, sw = product_inputs(rng, M, N, K, E)
    cut = cuts(M, E, kind)
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw), offsets=dev(cut), y=y)
    want, mag = ref.matmul(a, sa, w, sw, cut)
    check_product(y, want, mag, K, dtype)
    assert torch.all(y[int(cut[E]):] == 0)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("kind,dtype", list(zip(KINDS, [torch.float32, torch.bfloat16] * 2)))
@pytest.mark.parametrize("P,H,I,E", [(1500, 2576, 2576, 4), (4500, 2576, 1296, 3)])
def test_experts(P, H, I, E, kind, dtype):
    rng = np.random.default_rng(P + len(kind))
    t = expert_inputs(rng, P, H, I, E)
    cut = cuts(P, E, kind)
    a, sa, *weights = t
    y = torch.full((P, H), 3.0, dtype=dtype, device="cuda")
    zffn.fp8_experts(f8(a), f32(sa), *(f8(m) if i % 2 == 0 else f32(m) for i, m in enumerate(weights)), offsets=dev(cut), y=y)
    at = []
    for e in range(E):
        lo, hi = int(cut[e]), int(cut[e + 1])
        near = {lo, lo + 1, lo + 31, lo + 32, lo + 127, lo + 128, lo + 255, lo + 256, hi - 33, hi - 2, hi - 1, (lo + hi) // 2}
        at.append(sorted(r for r in near if lo <= r < hi))
    some = np.array([r for rows in at for r in rows])
    small = np.concatenate([[0], np.cumsum([len(rows) for rows in at])])
    want, tol = experts_ref(a[some], sa[some], *weights, small)
    if dtype == torch.bfloat16:
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(want)
    got = y[torch.from_numpy(some).cuda()].double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])
    assert torch.all(y[int(cut[E]):] == 0)
    assert zffn.get_device_error() == zffn.OK

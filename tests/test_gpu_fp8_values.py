"""Values at the ends of the range through the experts' fused epilogue: infinities and NaN among the gate
and up values, and gates whose silu is close to the smallest normal number.  On every kind of tile (16, 32
and 64 rows; single large tiles; CTA pairs).

The experts' h is seen through a down projection that picks features (one weight of 1 a row, scales 1), so
y is h's e4m3 value times its scale, exactly; a NaN in a row of h makes its whole row of y NaN."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import f8_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_fp8 import U32, f8, f32

pytestmark = pytest.mark.gpu

H = 64
# (rows, features, experts; 0: dense)
TILES = [(9, 528, 0), (40, 528, 2), (60, 656, 1), (1500, 2576, 4), (700, 9808, 0)]


def byte(v):
    return ref.to_byte(np.asarray(v, np.float64))


def picks(rng, I):
    """A down projection [H, I] of one 1 a row, and the features that it picks."""
    at = rng.integers(0, I, H)
    wd = np.zeros((H, I), np.uint8)
    wd[np.arange(H), at] = byte(1.0)
    return wd, at


def run(a, sa, wg, sg, wu, su, wd, E, P):
    """y of experts that all have these weights (dense: one)."""
    sd = np.ones((1, ref.blocks(wd.shape[1])), np.float32)
    parts = [wg, sg, wu, su, wd, sd]
    cut = None
    if E:
        parts = [np.repeat(t[None], E, 0) for t in parts]
        cut = dev(np.linspace(0, P, E + 1).astype(np.int32))
    t = [f8(p) if i % 2 == 0 else f32(p) for i, p in enumerate(parts)]
    y = zffn.fp8_experts(f8(a), f32(sa), *t, offsets=cut, dtype=torch.float32)
    assert zffn.get_device_error() == zffn.OK
    return y.double().cpu().numpy()


@pytest.mark.parametrize("P,I,E", TILES)
def test_infinities_and_nan_through_the_epilogue(P, I, E):
    # gate = a0 wg0 + a1 wg1 (one of the two is zero), so every product is exact or overflows; a gate beyond
    # 2^127 is +-inf in rows of scale 2^100; up values are 0 or powers of two, so a finite h has four
    # significant bits and its e4m3 value is h wherever the block's scale leaves it normal
    rng = np.random.default_rng(P + I)
    hot, second = rng.random(P) < 0.6, rng.random(P) < 0.3
    a = np.zeros((P, H), np.uint8)
    a[:, 0], a[second, 1] = byte(1.0), byte(1.0)
    sa = np.where(hot, 2.0 ** 100, 1.0)[:, None]
    wg, wu = np.zeros((I, H), np.uint8), np.zeros((I, H), np.uint8)
    kind = np.arange(ref.blocks(I)).repeat(128)[:I] % 4
    finite, some = [2.0 ** -6, 1.5 * 2.0 ** -5, 0.875, 96.0, 128.0, -1.0, 0.0], [448.0, 256.0, 1.0, 2.0 ** -6, 0.0]
    gate = np.where(kind == 0, rng.choice(finite, I), np.where(kind == 1, rng.choice(some, I), np.where(kind == 2, 448.0, 0.0)))
    minus = np.where(kind == 3, rng.choice([-448.0, 448.0, 0.0], I), 0.0)      # -inf (or inf times 0): NaN in the rows with a1
    up = np.where(kind == 3, rng.choice([0.0, 1.0], I), rng.choice([1.0, -1.0, 0.5, 2.0], I))
    wg[:, 0], wg[:, 1], wu[:, 0] = byte(gate), byte(minus), byte(up)
    one = np.ones((ref.blocks(I), 1))
    wd, at = picks(rng, I)
    y = run(a, sa, wg, 2.0 ** 20 * one, wu, 2.0 ** -100 * one, wd, E, P)
    with np.errstate(over="ignore", invalid="ignore"):
        g = ((gate[None] + second[:, None] * minus[None]) * (sa * 2.0 ** 20)).astype(np.float32)
        u = (up[None] * (sa * 2.0 ** -100)).astype(np.float32)
        h = (g / (1 + np.exp(-g.astype(np.float64)))).astype(np.float32) * u      # (fp32: may overflow)
        q, s = ref.quantize(h)
        v = ref.values(q, s)
    want = np.where(np.isnan(v).any(1)[:, None], np.nan, v[:, at])
    assert np.isinf(h).any() and np.isnan(want).any() and np.isfinite(want).any()
    assert (np.abs(want) == 448.0).any()                                        # blocks without a finite value: scale 1
    assert np.array_equal(y, want, equal_nan=True), (np.argwhere(~((y == want) | (np.isnan(y) & np.isnan(want))))[:5])


@pytest.mark.parametrize("P,I,E", TILES)
def test_gates_far_below_zero(P, I, E):
    # g = -G in the whole row, u = G 2^80 wu: h = silu(-G) u down to G = 87, with silu(-G) u off by at most
    # (3 + G / 3) 2^-22 of itself and u by two roundings; within that a byte may fall on the other side of a
    # border.  Beyond 87.4 silu is 0.
    rng = np.random.default_rng(P * I)
    G = rng.choice([0.5, 1.0, 5.0, 20.0, 40.0, 60.0, 80.0, 86.9, 87.3, 87.4, 88.0, 100.0, 1e4, 1e8], P).astype(np.float32)
    a = np.zeros((P, H), np.uint8)
    a[:, 0] = byte(1.0)
    wg, wu = np.zeros((I, H), np.uint8), np.zeros((I, H), np.uint8)
    wg[:, 0], wu[:, 0] = byte(-1.0), ref.random_e4m3(rng, I)
    one = np.ones((ref.blocks(I), 1))
    wd, at = picks(rng, I)
    y = run(a, G[:, None], wg, one, wu, 2.0 ** 80 * one, wd, E, P)
    g = -G.astype(np.float64)[:, None]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    h = silu * (-g * 2.0 ** 80 * ref.VALUES[wu[:, 0]][None])
    h[G > 87.35] = 0.0
    eh = np.abs(h) * ((3 + np.abs(g) / 3) * 2.0 ** -22 + 2 * U32)
    v, lo, hi = (ref.values(*ref.quantize(t)) for t in (h, h - eh, h + eh))
    flip = np.maximum(np.abs(lo - v), np.abs(hi - v))
    assert np.all(np.abs(y - v[:, at]) <= flip[:, at])
    assert np.all(y[G > 87.35] == 0) and np.all((y[G < 87] != 0).any(1))

"""The block-scaled e4m3 operators (quantise, dequantise, products, experts) against plain 64-bit
forms, through the public Python entry points.

Tolerances.  Quantisation: x / s is exact and rounded once, so bytes and scales must be equal.
Products: every a*w product is exact in fp32 (two 4-bit significands); what rounds are the sums of
a block (128 terms), the scales' product (1), its product with the block's sum and the sum over
ceil(K/128) blocks.  Each of those steps is off by at most 2^-24 of a partial sum, itself at most
the sum of magnitudes; the tensor cores may cut instead of round and align a group of terms to its
largest, so a block's sum is allowed 4 * 2^-24 for each of its 4 groups of 32: in all
(16 + 2 + 2 * blocks) * 2^-24 of `mag`.  A bf16 result adds half a step, 2^-8 of the value
(eps / 2), as the final rounding."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import f8_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def f8(b):
    return dev(b).view(torch.float8_e4m3fn)


def f32(a):
    return dev(np.asarray(a, np.float32))


def check_product(y, want, mag, K, dtype):
    tol = (16 + 2 + 2 * ref.blocks(K)) * U32 * mag
    if dtype == torch.bfloat16:
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(want)
    got = y.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


# ---- quantise, dequantise -------------------------------------------------------------------

@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (37, 1040), (5, 7), (130, 264), (129, 4096), (64, 2049)])
def test_quantize_is_exact(rows, cols, dtype, block_rows):
    rng = np.random.default_rng(rows * 131 + cols)
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-6, 6, (rows, 1))
    x[rng.random((rows, cols)) < 0.1] = 0.0
    t = dev(x.astype(np.float32)).to(dtype)
    q, s = zffn.fp8_quantize(t, block_rows=block_rows)
    wq, ws = ref.quantize(t.double().cpu().numpy(), block_rows)
    assert np.array_equal(s.double().cpu().numpy(), ws)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), wq)
    back = zffn.fp8_dequant(q, s, block_rows=block_rows)
    assert np.array_equal(back.double().cpu().numpy(), ref.values(wq, ws, block_rows))


def test_quantize_at_the_borders():
    # 448 * 2^p exactly and one step above, zeros, the smallest and largest fp32, inf and NaN
    f = np.float32
    rows = [[448.0, 1.0], [np.nextafter(f(448), f(1e9)), 1.0], [0.0, -0.0], [1e-45, 0.0], [3.4028235e38, -1.0],
            [np.inf, 3.0], [np.nan, -7.0], [-np.inf, 0.0], [np.nan, np.nan], [2.0 ** -130, 2.0 ** -140], [17.0, 19.0]]
    x = np.zeros((len(rows), 130), np.float32)
    x[:, [0, 127]] = np.array(rows, np.float32)
    x[:, 128:] = x[:, [127, 0]]
    for block_rows in (1, 128):
        q, s = zffn.fp8_quantize(dev(x), block_rows=block_rows)
        wq, ws = ref.quantize(x, block_rows)
        assert np.array_equal(s.double().cpu().numpy(), ws)
        got = q.view(torch.uint8).cpu().numpy()
        nan = np.isnan(x)
        assert np.all((got[nan] & 0x7F) == 0x7F)
        assert np.array_equal(got[~nan], wq[~nan])


def test_quantize_of_unaligned_rows():
    rng = np.random.default_rng(3)
    for off in (1, 2, 4):
        x = torch.zeros(off + 5 * 256, dtype=torch.bfloat16, device="cuda")
        x[off:] = dev(rng.standard_normal(5 * 256).astype(np.float32))
        t = x[off:].view(5, 256)
        q, s = zffn.fp8_quantize(t)
        wq, ws = ref.quantize(t.double().cpu().numpy())
        assert np.array_equal(q.view(torch.uint8).cpu().numpy(), wq) and np.array_equal(s.double().cpu().numpy(), ws)


def test_every_byte_dequantizes():
    b = np.tile(np.arange(256, dtype=np.uint8), (2, 1))
    out = zffn.fp8_dequant(f8(b), f32([[1.0, 2.0], [0.3, 1e-3]])).double().cpu().numpy()
    s = np.float32([[1.0, 2.0], [0.3, 1e-3]]).astype(np.float64)
    want = ref.values(b, s)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(out), nan)
    np.testing.assert_allclose(out[~nan], want[~nan], rtol=U32, atol=0)


# ---- products -------------------------------------------------------------------------------

def product_inputs(rng, M, N, K, E=0):
    lead = (E,) if E else ()
    a, w = ref.random_e4m3(rng, (M, K)), ref.random_e4m3(rng, (*lead, N, K))
    sa = np.exp(rng.uniform(-3, 3, (M, ref.blocks(K)))).astype(np.float32)
    sw = np.exp(rng.uniform(-7, -1, (*lead, ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    return a, sa, w, sw


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 2057, 1040), (2, 130, 144), (7, 64, 16), (16, 129, 4096), (17, 256, 400),
          (33, 300, 1040), (64, 1000, 512), (65, 384, 272), (100, 129, 2064), (128, 256, 256), (129, 257, 272),
          (200, 512, 1024), (256, 1024, 384), (300, 2049, 528), (513, 768, 1152), (130, 10001, 272), (255, 9728, 144),
          (256, 9999, 400), (700, 4096, 272), (1030, 2568, 1040), (2500, 1032, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense_product(M, N, K, dtype):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    a, sa, w, sw = product_inputs(rng, M, N, K)
    y = zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw), dtype=dtype)
    want, mag = ref.matmul(a, sa, w, sw)
    check_product(y, want, mag, K, dtype)
    assert zffn.get_device_error() == zffn.OK


def split_rows(rng, M, E, kind):
    if kind == "one":        # every row to one expert
        cut = np.zeros(E + 1, np.int32)
        cut[E // 2 + 1:] = M
    elif kind == "unused":   # a third of the rows belong to no expert
        cut = np.sort(rng.integers(0, 2 * M // 3 + 1, E + 1)).astype(np.int32)
        cut[0] = 0
    else:                    # random, many experts empty when E is large
        cut = np.sort(rng.integers(0, M + 1, E + 1)).astype(np.int32)
        cut[0], cut[E] = 0, M
    return cut


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["random", "one", "unused"])
@pytest.mark.parametrize("M,N,K,E", [(1, 136, 144, 5), (8, 256, 256, 128), (40, 130, 400, 3), (100, 200, 272, 40),
                                     (300, 384, 528, 2), (700, 257, 144, 5), (1500, 256, 256, 4)])
def test_grouped_product(M, N, K, E, kind, dtype):
    rng = np.random.default_rng(M + 100 * E + len(kind))
    a, sa, w, sw = product_inputs(rng, M, N, K, E)
    cut = split_rows(rng, M, E, kind)
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw), offsets=dev(cut), y=y)
    want, mag = ref.matmul(a, sa, w, sw, cut)
    check_product(y, want, mag, K, dtype)
    assert torch.all(y[int(cut[E]):] == 0)


@pytest.mark.parametrize("M,E", [(3, 4096), (5000, 4096)])
def test_grouped_product_of_many_experts(M, E):
    rng = np.random.default_rng(M)
    a, sa, w, sw = product_inputs(rng, M, 16, 16, E)
    cut = split_rows(rng, M, E, "random")
    y = zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw), offsets=dev(cut))
    want, mag = ref.matmul(a, sa, w, sw, cut)
    check_product(y, want, mag, 16, torch.float32)


def test_nan_and_zero_rows_stay_in_their_rows():
    rng = np.random.default_rng(5)
    for M, N in ((5, 200), (140, 512)):
        a, sa, w, sw = product_inputs(rng, M, N, 272)
        a[1, 3] = 0x7F
        a[2] = 0
        w[7, 270] = 0xFF
        y = zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw)).double().cpu().numpy()
        nan = np.zeros((M, N), bool)
        nan[1] = True
        nan[:, 7] = True
        assert np.array_equal(np.isnan(y), nan)
        assert np.all(y[2][~nan[2]] == 0)


def test_product_into_unaligned_and_odd_outputs():
    rng = np.random.default_rng(9)
    for M, N, dtype in ((20, 255, torch.bfloat16), (150, 256, torch.bfloat16), (150, 256, torch.float32), (9, 128, torch.float32)):
        a, sa, w, sw = product_inputs(rng, M, N, 256)
        buf = torch.zeros(1 + M * N + 1, dtype=dtype, device="cuda")
        y = buf[1:1 + M * N].view(M, N)
        zffn.fp8_matmul(f8(a), f32(sa), f8(w), f32(sw), y=y)
        check_product(y, *ref.matmul(a, sa, w, sw), 256, dtype)
        assert buf[0] == 0 and buf[-1] == 0


def test_product_is_the_same_every_time():
    rng = np.random.default_rng(11)
    for M, N, K in ((3, 1000, 4096), (300, 512, 2048)):
        a, sa, w, sw = (t for t in product_inputs(rng, M, N, K))
        t = (f8(a), f32(sa), f8(w), f32(sw))
        first = zffn.fp8_matmul(*t)
        for _ in range(5):
            assert torch.equal(first, zffn.fp8_matmul(*t))


def test_gradient_by_the_input_is_the_product_on_transposed_weights():
    # d/da of sum(g * y), y = a W^T, is g W; against the formula in 64 bits and against differences of y
    rng = np.random.default_rng(13)
    M, N, K = 24, 272, 400
    a, sa, w, sw = product_inputs(rng, M, N, K)
    g = rng.standard_normal((M, N)).astype(np.float32)
    gq, gs = zffn.fp8_quantize(dev(g))
    wt = np.ascontiguousarray(w.T)
    dx = zffn.fp8_matmul(gq, gs, f8(wt), f32(np.ascontiguousarray(sw.T)))
    gv = ref.values(gq.view(torch.uint8).cpu().numpy(), gs.cpu().numpy())
    wv = ref.values(w, sw, 128)
    check_product(dx, gv @ wv, np.abs(gv) @ np.abs(wv), N, torch.float32)
    # y is linear in a: one step of one input value moves sum(g * y) by step * gradient
    x = ref.values(a, sa)
    m, k = 5, 301
    step = x.copy()
    step[m, k] += 1.0
    diff = (gv * (step @ wv.T - x @ wv.T)).sum()
    assert abs(diff - float(dx[m, k])) <= 1e-4 * (np.abs(gv[m]) * np.abs(wv[:, k])).sum()


def test_product_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(17)
    for M, N, K in ((4, 300, 1040), (260, 512, 528)):
        a, sa, w, sw = product_inputs(rng, M, N, K)
        t = (f8(a), f32(sa), f8(w), f32(sw))
        want = zffn.fp8_matmul(*t)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y = torch.zeros_like(want)
        with torch.cuda.stream(s):
            zffn.fp8_matmul(*t, y=y)
        s.synchronize()
        assert torch.equal(y, want)
        g = torch.cuda.CUDAGraph()
        y.zero_()
        with torch.cuda.graph(g):
            zffn.fp8_matmul(*t, y=y)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ---- experts --------------------------------------------------------------------------------

def expert_inputs(rng, P, H, I, E):
    a = ref.random_e4m3(rng, (P, H))
    sa = (2.0 ** rng.integers(-7, -4, (P, ref.blocks(H)))).astype(np.float32)
    out = [a, sa]
    lead = (E,) if E else ()
    for n, k in ((I, H), (I, H), (H, I)):
        out.append(ref.random_e4m3(rng, (*lead, n, k)))
        out.append((rng.uniform(0.3, 1.0, (*lead, ref.blocks(n), ref.blocks(k))) * 0.05 / 40).astype(np.float32))
    return out


def experts_ref(a, sa, wg, sg, wu, su, wd, sd, cut):
    """y in 64 bits, and a bound of its error: h's fp32 value is off by at most eh (the products' bound
    carried through silu(g) u, |silu'| <= 1.1, and 8 steps of the exponential and the division); near a
    border of e4m3 (or of its scale) the byte may then fall on either side, so every h within eh of a
    border may be one e4m3 step (2^-3 of the value, 2 half steps) off, the others are equal."""
    P, H = a.shape
    E, I = wg.shape[0], wg.shape[1]
    y, tol = np.zeros((P, H)), np.zeros((P, H))
    for e in range(E):
        at = slice(int(cut[e]), int(cut[e + 1]))
        if at.start == at.stop:
            continue
        g, gm = ref.matmul(a[at], sa[at], wg[e], sg[e])
        u, um = ref.matmul(a[at], sa[at], wu[e], su[e])
        c = (18 + 2 * ref.blocks(H)) * U32
        silu = g / (1 + np.exp(-g))
        h = silu * u
        eh = c * (1.1 * gm * np.abs(u) + np.abs(silu) * um) + 8 * U32 * np.abs(h) * (1 + np.abs(g) / 4)
        q, s = ref.quantize(h)
        ql, sl = ref.quantize(h - eh)
        qh, sh = ref.quantize(h + eh)
        v = ref.values(q, s)
        flip = np.maximum(np.abs(ref.values(ql, sl) - v), np.abs(ref.values(qh, sh) - v))
        wv = np.abs(ref.values(wd[e], sd[e], 128))
        y[at] = v @ ref.values(wd[e], sd[e], 128).T
        tol[at] = (18 + 2 * ref.blocks(I)) * U32 * (np.abs(v) @ wv.T) + flip @ wv.T
    return y, tol


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("P,H,I,E,kind", [(1, 256, 128, 1, "random"), (8, 512, 192, 16, "random"), (40, 272, 144, 3, "unused"),
                                          (64, 256, 16, 2, "one"), (130, 384, 768, 4, "random"), (400, 256, 272, 2, "random"),
                                          (900, 512, 256, 3, "unused"), (1300, 256, 400, 4, "one")])
def test_experts(P, H, I, E, kind, dtype):
    rng = np.random.default_rng(P + H + I)
    t = expert_inputs(rng, P, H, I, E)
    cut = split_rows(rng, P, E, kind)
    a, sa, wg, sg, wu, su, wd, sd = t
    y = torch.full((P, H), 3.0, dtype=dtype, device="cuda")
    zffn.fp8_experts(f8(a), f32(sa), f8(wg), f32(sg), f8(wu), f32(su), f8(wd), f32(sd), offsets=dev(cut), y=y)
    want, tol = experts_ref(*t, cut)
    if dtype == torch.bfloat16:
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(want)
    got = y.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])
    assert np.abs(want).max() > 0
    # the dense form is expert 0 alone
    if E == 1:
        d = zffn.fp8_experts(f8(a), f32(sa), f8(wg[0]), f32(sg[0]), f8(wu[0]), f32(su[0]), f8(wd[0]), f32(sd[0]), dtype=dtype)
        assert torch.equal(d, y)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("P,H,I,kind", [(700, 256, 9808, "random"), (200, 272, 9744, "unused")])
def test_experts_of_large_tiles(P, H, I, kind):
    # wide enough that the dense gate/up product fills the SMs with large tiles, its down product not;
    # one expert's grouped form may take other tiles, so each is held to the bound
    rng = np.random.default_rng(P + H + I)
    t = expert_inputs(rng, P, H, I, 1)
    cut = split_rows(rng, P, 1, kind)
    a, sa, wg, sg, wu, su, wd, sd = t
    for offsets in (dev(cut), None):
        if offsets is None:
            y = zffn.fp8_experts(f8(a), f32(sa), f8(wg[0]), f32(sg[0]), f8(wu[0]), f32(su[0]), f8(wd[0]), f32(sd[0]), dtype=torch.float32)
            want, tol = experts_ref(*t, np.array([0, P]))
        else:
            y = zffn.fp8_experts(f8(a), f32(sa), f8(wg), f32(sg), f8(wu), f32(su), f8(wd), f32(sd), offsets=offsets, dtype=torch.float32)
            want, tol = experts_ref(*t, cut)
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol + 1e-37)


@pytest.mark.parametrize("P,H,I,E", [(12000, 144, 32, 1000), (3000, 32, 16, 4096), (130000, 32, 16, 4096)])
def test_experts_of_many_experts(P, H, I, E):
    # the table of the experts' rows takes shared memory beside the tiles
    rng = np.random.default_rng(P + E)
    t = expert_inputs(rng, P, H, I, E)
    cut = split_rows(rng, P, E, "random")
    a, sa, wg, sg, wu, su, wd, sd = t
    y = zffn.fp8_experts(f8(a), f32(sa), f8(wg), f32(sg), f8(wu), f32(su), f8(wd), f32(sd), offsets=dev(cut), dtype=torch.float32)
    want, tol = experts_ref(*t, cut)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol + 1e-37)
    assert zffn.get_device_error() == zffn.OK


def test_routed_layer_end_to_end():
    # router -> routed block against the oracle's router and the steps in 64 bits; the sum over slots
    # adds the bf16 rows' half step and k fp32 steps
    rng = np.random.default_rng(21)
    for T, H, I, E, k in ((1, 256, 128, 16, 4), (50, 512, 256, 8, 3), (300, 256, 144, 4, 2)):
        x = torch.randn((T, H), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
        logits = dev(rng.standard_normal((T, E)).astype(np.float32))
        ids, w = zffn.moe_router_topk(logits, k)
        _, _, wg, sg, wu, su, wd, sd = expert_inputs(rng, 1, H, I, E)
        args = (f8(wg), f32(sg), f8(wu), f32(su), f8(wd), f32(sd))
        y = zffn.moe_swiglu_fp8(x.cuda(), ids, w, *args)
        q, s = ref.quantize(x.double().numpy())
        row_slot, slot_row, cut = ref.sort(ids.cpu().numpy(), E)
        rows, tol = experts_ref(q[row_slot // k], s[row_slot // k], wg, sg, wu, su, wd, sd, cut)
        wn = w.double().cpu().numpy()
        want, bound = np.zeros((T, H)), np.zeros((T, H))
        for j in range(k):
            r, e = rows[slot_row[:, j]], tol[slot_row[:, j]]
            want += wn[:, j, None] * r
            bound += wn[:, j, None] * (e * (1 + HALF_BF16) + (HALF_BF16 + 2 * k * U32) * np.abs(r))
        got = y.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= bound + 1e-37)
        # the same steps one by one, and the residual form
        qx, sx = zffn.fp8_quantize(x.cuda())
        plan = zffn.moe_sort(ids, E)
        xs, ss = zffn.moe_dispatch(qx, plan, scale=sx)
        r = zffn.fp8_experts(xs, ss, *args, offsets=plan.offsets)
        assert torch.equal(zffn.moe_combine(r, plan, w), y)
        res = torch.ones_like(y)
        zffn.moe_swiglu_fp8(x.cuda(), ids, w, *args, y=res, accumulate=True)
        torch.testing.assert_close(res, y + 1, rtol=4 * k * U32, atol=4 * k * U32)

"""The sort by expert, the rows' way to their sorted places and back, and the gradients, against
plain forms.  The sort and the copies are exact.  Sums over slots: k products and additions in
fp32, each off by at most 2^-24 of the sum of magnitudes; dot products over H in fp32 with at
most H / 32 + 5 additions in a chain (a lane's share, then the warp), each 2^-24 of the sum of
magnitudes; bf16 gradients add half a step (2^-8 of the value)."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import f8_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def make_ids(rng, T, E, k, kind):
    if kind == "one":
        return np.full((T, k), E // 2, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "skewed":
        ids = np.minimum(rng.geometric(0.2, (T, k)) - 1, E - 1).astype(np.int32)
    if kind == "dropped":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E
        ids[0, 0] = np.iinfo(np.int32).min
    return ids


@pytest.mark.parametrize("kind", ["random", "one", "none", "skewed", "dropped"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 7, 64), (31, 128, 1), (33, 4096, 5), (128, 60, 8), (129, 128, 8),
                                   (1025, 128, 8), (4096, 128, 8), (5000, 3, 2), (3001, 4096, 7), (70000, 33, 3)])
def test_sort(T, E, k, kind):
    rng = np.random.default_rng(T + E + k)
    ids = make_ids(rng, T, E, k, kind)
    plan = zffn.moe_sort(dev(ids), E)
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    used = int((key < E).sum())
    row_slot = np.where(np.arange(T * k) < used, order, -1)
    slot_row = np.full(T * k, -1)
    slot_row[order[:used]] = np.arange(used)
    assert np.array_equal(plan.offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(E + 1)))
    assert np.array_equal(plan.row_slot.cpu().numpy(), row_slot)
    assert np.array_equal(plan.slot_row.cpu().numpy().reshape(-1), slot_row)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.float64])
@pytest.mark.parametrize("T,E,k,H", [(1, 128, 8, 2048), (5, 4, 3, 1), (37, 60, 5, 1041), (64, 8, 2, 4096), (33, 3, 64, 130)])
def test_dispatch_copies_rows(T, E, k, H, dtype):
    rng = np.random.default_rng(H)
    ids = make_ids(rng, T, E, k, "dropped")
    plan = zffn.moe_sort(dev(ids), E)
    x = dev(rng.integers(0, 250, (T, H)).astype(np.float64)).to(dtype)
    out = torch.full((T * k, H), 9, device="cuda").to(dtype)
    zffn.moe_dispatch(x, plan, out=out)
    row_slot, _, _ = ref.sort(ids, E)
    want = np.where((row_slot >= 0)[:, None], x.double().cpu().numpy()[np.maximum(row_slot, 0) // k], 0.0)
    assert np.array_equal(out.double().cpu().numpy(), want)


def test_dispatch_of_scales_and_unaligned_rows():
    rng = np.random.default_rng(2)
    T, E, k, H = 29, 6, 4, 272
    ids = make_ids(rng, T, E, k, "dropped")
    plan = zffn.moe_sort(dev(ids), E)
    row_slot, _, _ = ref.sort(ids, E)
    at, live = np.maximum(row_slot, 0) // k, (row_slot >= 0)[:, None]
    buf = dev(rng.integers(0, 256, 3 + T * H).astype(np.uint8))
    s = dev(rng.standard_normal((T, 3)).astype(np.float32))
    for off in (0, 1, 2, 3):
        x = buf[off:off + T * H].view(T, H)
        xs, ss = zffn.moe_dispatch(x, plan, scale=s)
        assert np.array_equal(xs.cpu().numpy(), np.where(live, x.cpu().numpy()[at], 0))
        assert np.array_equal(ss.cpu().numpy(), np.where(live, s.cpu().numpy()[at], 0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["random", "dropped", "none"])
@pytest.mark.parametrize("T,E,k,H", [(1, 128, 8, 2048), (5, 4, 3, 1), (37, 60, 5, 1041), (50, 8, 2, 4096), (9, 3, 64, 130), (300, 16, 8, 512),
                                     (7, 5, 3, 2026), (3, 2, 2, 9001), (2, 2, 1, 65536)])
def test_combine_and_gradients(T, E, k, H, kind, dtype):
    rng = np.random.default_rng(T + H)
    ids = make_ids(rng, T, E, k, kind)
    plan = zffn.moe_sort(dev(ids), E)
    row_slot, slot_row, _ = ref.sort(ids, E)
    rows_t = dev(rng.standard_normal((T * k, H)).astype(np.float32)).to(dtype)
    w_t, dy_t = dev(rng.random((T, k)).astype(np.float32)), dev(rng.standard_normal((T, H)).astype(np.float32))
    rows, w, dy = (t.double().cpu().numpy() for t in (rows_t, w_t, dy_t))
    live = (slot_row >= 0)[..., None]
    got_rows = np.where(live, rows[np.maximum(slot_row, 0)], 0.0)          # [T, k, H]

    y = zffn.moe_combine(rows_t, plan, w_t).double().cpu().numpy()
    want, mag = (got_rows * w[..., None]).sum(1), (np.abs(got_rows) * w[..., None]).sum(1)
    assert np.all(np.abs(y - want) <= 2 * k * U32 * mag)
    base = dev(rng.standard_normal((T, H)).astype(np.float32))
    z = zffn.moe_combine(rows_t, plan, w_t, y=base.clone(), accumulate=True).double().cpu().numpy()
    b = base.double().cpu().numpy()
    assert np.all(np.abs(z - (b + want)) <= 2 * (k + 1) * U32 * (mag + np.abs(b)))
    dx = zffn.moe_combine(rows_t, plan, None).double().cpu().numpy()
    assert np.all(np.abs(dx - got_rows.sum(1)) <= 2 * k * U32 * np.abs(got_rows).sum(1))

    drows, dw = zffn.moe_combine_grad(dy_t, rows_t, plan, w_t)
    wr = np.where((row_slot >= 0)[:, None], w.reshape(-1)[np.maximum(row_slot, 0)][:, None] * dy[np.maximum(row_slot, 0) // k], 0.0)
    half = HALF_BF16 if dtype == torch.bfloat16 else 0.0
    assert drows.dtype == dtype
    assert np.all(np.abs(drows.double().cpu().numpy() - wr) <= (U32 * (1 + half) + half) * np.abs(wr) + 1e-40)
    dwant, dmag = (got_rows * dy[:, None]).sum(2), np.abs(got_rows * dy[:, None]).sum(2)
    assert np.all(np.abs(dw.double().cpu().numpy() - dwant) <= 2 * (H / 32 + 5) * U32 * dmag)
    # differences: y is linear in rows and in weights, so a step of one moves <dy, y> by the gradient
    # (to the rounding of y's own fp32 sums)
    if kind == "random":
        t, j = T // 2, k - 1
        w2 = w_t.clone()
        w2[t, j] += 1.0
        y2 = zffn.moe_combine(rows_t, plan, w2).double().cpu().numpy()
        step = float(w2[t, j].double() - w_t[t, j].double())
        tol = 2 * k * U32 * (np.abs(dy[t]) * (2 * mag[t] + np.abs(got_rows[t, j]))).sum() + 2 * (H / 32 + 5) * U32 * dmag[t, j]
        assert abs((dy[t] * (y2 - y)[t]).sum() - step * float(dw[t, j])) <= tol
    # either output alone
    only, none = torch.empty_like(drows), torch.empty_like(dw)
    lib, p = zffn.load(), lambda a: a.data_ptr()
    args = (p(plan.row_slot), p(plan.slot_row), p(w_t))
    d = zffn.DT_BF16 if dtype == torch.bfloat16 else zffn.DT_F32
    assert lib.zffn_moe_combine_grad(d, p(dy_t), None, *args, p(only), None, T, H, k, None) == zffn.OK
    assert lib.zffn_moe_combine_grad(d, p(dy_t), p(rows_t), args[0], args[1], None, None, p(none), T, H, k, None) == zffn.OK
    torch.cuda.synchronize()
    assert torch.equal(only, drows) and torch.equal(none, dw)


def test_unaligned_rows_combine():
    rng = np.random.default_rng(6)
    T, E, k, H = 17, 4, 2, 256
    ids = make_ids(rng, T, E, k, "random")
    plan = zffn.moe_sort(dev(ids), E)
    w = dev(rng.random((T, k)).astype(np.float32))
    dy = dev(rng.standard_normal((T, H)).astype(np.float32))
    buf = dev(rng.standard_normal(1 + T * k * H).astype(np.float32)).to(torch.bfloat16)
    odd = buf[1:].view(T * k, H)
    even = odd.clone()
    assert torch.equal(zffn.moe_combine(odd, plan, w), zffn.moe_combine(even, plan, w))
    a, b = zffn.moe_combine_grad(dy, odd, plan, w, drows=torch.empty_like(even)), zffn.moe_combine_grad(dy, even, plan, w)
    assert torch.equal(a[0], b[0])
    torch.testing.assert_close(a[1], b[1], rtol=1e-4, atol=1e-4)


def test_weights_of_special_values():
    # a pair without a row takes no part, whatever its weight; a weight of 0 times inf is NaN as in fp32
    plan = zffn.moe_sort(dev(np.array([[0, -1], [1, 0]], np.int32)), 2)
    rows = torch.ones((4, 8), device="cuda")
    rows[int(plan.slot_row[1, 0])] = float("inf")
    w = dev(np.array([[2.0, np.nan], [0.0, 1.0]], np.float32))
    y = zffn.moe_combine(rows, plan, w)
    assert torch.all(y[0] == 2.0) and torch.all(torch.isnan(y[1]))
    _, dw = zffn.moe_combine_grad(torch.ones((2, 8), device="cuda"), rows, plan, w)
    assert dw[0, 1] == 0 and torch.isinf(dw[1, 0])


def test_sort_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(8)
    T, E, k, H = 700, 32, 4, 256
    ids = dev(make_ids(rng, T, E, k, "random"))
    x = dev(rng.standard_normal((T, H)).astype(np.float32))
    w = torch.full((T, k), 0.25, device="cuda")
    zffn.moe_sort(ids, E)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan = zffn.moe_sort(ids, E)
        y = zffn.moe_combine(zffn.moe_dispatch(x, plan), plan, w)
    ids.copy_(dev(make_ids(rng, T, E, k, "skewed")))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, x)          # four quarters of the row, exact in fp32
    assert np.array_equal(plan.row_slot.cpu().numpy(), ref.sort(ids.cpu().numpy(), E)[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = zffn.moe_sort(ids, E)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, plan))


def test_plan_parts_outlive_each_other():
    # the three parts of a new plan are one allocation, which lives as long as any of them
    rng = np.random.default_rng(23)
    T, E, k = 37, 12, 3
    ids = make_ids(rng, T, E, k, "random")
    want = ref.sort(ids, E)
    for keep in range(3):
        part = zffn.moe_sort(dev(ids), E)[keep]
        assert part.is_contiguous() and part.dtype == torch.int32 and part.shape == want[keep].shape
        torch.full((2 * T * k + 64,), -9, dtype=torch.int32, device="cuda")
        assert np.array_equal(part.cpu().numpy(), want[keep])
        copy = part.clone()
        part += 1
        assert torch.equal(part, copy + 1)

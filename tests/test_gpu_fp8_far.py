"""The 8-bit and sorting operators on arrays of more than 2^31 elements (or 2^32 bytes): rows from both
ends and from either side of the 2^31st element, against the same rows on their own or in 64 bits.
Tolerances as in test_gpu_fp8.py and test_gpu_moe_sort.py."""
import numpy as np
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import f8_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_fp8 import HALF_BF16, U32, check_product, experts_ref, f32, f8, product_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def some_rows(rows, cols):
    edge = 2 ** 31 // cols
    assert edge + 1 < rows - 3
    return np.array([0, 1, edge - 1, edge, edge + 1, 2 * edge // 3, rows - 3, rows - 2, rows - 1])


@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 8192), (torch.bfloat16, 8203), (torch.float32, 8200)])
def test_quantise(dtype, cols):
    rows = 2 ** 31 // cols + 700
    x = torch.empty((rows, cols), dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(cols))
    q, s = zffn.fp8_quantize(x)
    at = torch.from_numpy(some_rows(rows, cols)).cuda()
    q1, s1 = zffn.fp8_quantize(x[at].contiguous())
    assert torch.equal(q.view(torch.uint8)[at], q1.view(torch.uint8)) and torch.equal(s[at], s1)
    d = zffn.fp8_dequant(q, s)
    assert torch.equal(d[at], zffn.fp8_dequant(q1, s1))


def far_weights(rng, E, N, K):
    gen = torch.Generator(device="cuda").manual_seed(N + E)
    w = torch.randint(0, 0x7F, (E, N, K), dtype=torch.uint8, device="cuda", generator=gen)   # (not negative, no NaN)
    sw = np.exp(rng.uniform(-7, -1, (E, ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    return w.view(torch.float8_e4m3fn), sw


@pytest.mark.parametrize("N,E,dtype", [(16400, 0, torch.bfloat16), (16401, 0, torch.float32), (16400, 4096, torch.bfloat16)])
def test_product(N, E, dtype):
    # large tiles (their stores by TMA, and by the lanes), and small ones
    M, K = 2 ** 31 // N + 500, 16
    rng = np.random.default_rng(N + E)
    a, sa, _, _ = product_inputs(rng, M, 16, K)
    w, sw = far_weights(rng, max(E, 1), N, K)
    cut = np.linspace(0, M, E + 1).astype(np.int32) if E else None
    y = zffn.fp8_matmul(f8(a), f32(sa), w if E else w[0], f32(sw if E else sw[0]), offsets=dev(cut) if E else None, dtype=dtype)
    for r in some_rows(M, N):
        e = int(np.searchsorted(cut, r, side="right")) - 1 if E else 0
        want, mag = ref.matmul(a[r:r + 1], sa[r:r + 1], w[e].view(torch.uint8).cpu().numpy(), sw[e])
        check_product(y[r:r + 1], want, mag, K, dtype)
    assert zffn.get_device_error() == zffn.OK


def test_product_of_far_weights():
    E, N, K, M = 64, 16400, 4112, 8
    rng = np.random.default_rng(9)
    a, sa, _, _ = product_inputs(rng, M, 16, K)
    w, sw = far_weights(rng, E, N, K)
    cut = np.zeros(E + 1, np.int32)
    cut[E // 2:] = 3      # three rows to the expert before the middle, five to the last
    cut[E] = M
    y = zffn.fp8_matmul(f8(a), f32(sa), w, f32(sw), offsets=dev(cut))
    for e, rows in ((E // 2 - 1, slice(0, 3)), (E - 1, slice(3, M))):
        want, mag = ref.matmul(a[rows], sa[rows], w[e].view(torch.uint8).cpu().numpy(), sw[e])
        check_product(y[rows], want, mag, K, torch.float32)


def test_experts():
    P, H, I = 2 ** 31 // 16384 + 500, 16, 16384
    rng = np.random.default_rng(5)
    t = [ref.random_e4m3(rng, (P, H)), np.exp(rng.uniform(-1, 1, (P, 1))).astype(np.float32)]
    for n, k in ((I, H), (I, H), (H, I)):
        t += [ref.random_e4m3(rng, (1, n, k)), (rng.uniform(0.3, 1.0, (1, ref.blocks(n), ref.blocks(k))) * 0.05 / 40).astype(np.float32)]
    a, sa, wg, sg, wu, su, wd, sd = t
    y = zffn.fp8_experts(f8(a), f32(sa), f8(wg[0]), f32(sg[0]), f8(wu[0]), f32(su[0]), f8(wd[0]), f32(sd[0]), dtype=torch.float32)
    at = some_rows(P, I)
    want, tol = experts_ref(a[at], sa[at], wg, sg, wu, su, wd, sd, np.array([0, len(at)]))
    assert np.all(np.abs(y[torch.from_numpy(at).cuda()].double().cpu().numpy() - want) <= tol + 1e-37)
    assert zffn.get_device_error() == zffn.OK
    zffn.release()   # (h's gigabytes)


@pytest.mark.parametrize("H", [8192, 8203])
def test_rows_to_their_places_and_back(H):
    k, E = 8, 64
    T = 2 ** 31 // (8 * H) + 100
    gen = torch.Generator(device="cuda").manual_seed(H)
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda", generator=gen)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.rand((T, k), device="cuda", generator=gen)
    plan = zffn.moe_sort(ids, E)
    rows = zffn.moe_dispatch(x, plan)
    used = int(plan.offsets[E])
    at = some_rows(T * k, H)
    for r in [int(v) for v in at] + [used - 1, used]:
        f = int(plan.row_slot[r])
        assert torch.equal(rows[r], x[f // k] if f >= 0 else torch.zeros_like(x[0]))
        assert (f < 0) == (r >= used)
    rows.normal_(generator=gen)
    y = zffn.moe_combine(rows, plan, w)
    dy = torch.empty((T, H), device="cuda").normal_(generator=gen)
    drows, dw = zffn.moe_combine_grad(dy, rows, plan, w)
    tokens = {0, T - 1, T // 2} | {int(plan.row_slot[r]) // k for r in at if int(plan.row_slot[r]) >= 0}
    for t in tokens:
        want, mag = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
        for j in range(k):
            r = int(plan.slot_row[t, j])
            if r < 0:
                assert float(dw[t, j]) == 0
                continue
            v, g = rows[r].double(), dy[t].double()
            want += w[t, j].double() * v
            mag += w[t, j].double() * v.abs()
            assert abs(float(dw[t, j]) - float((v * g).sum())) <= 2 * (H / 32 + 5) * U32 * float((v * g).abs().sum())
            wr = w[t, j].double() * g
            assert bool(((drows[r].double() - wr).abs() <= (U32 * (1 + HALF_BF16) + HALF_BF16) * wr.abs() + 1e-40).all())
        assert bool(((y[t].double() - want).abs() <= 2 * k * U32 * mag).all())
    assert used < T * k and not bool(drows[used:].any())

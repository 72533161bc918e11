"""bf16 products, dense and grouped by expert, and their gradients by input and weights, against 64-bit forms
(tests/bf16_ref.py, which derives the tolerances)."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
KINDS = ["random", "one", "none", "unused", "borders"]


def run_product(M, N, K, E, kind, transposed, dtype, seed=0):
    gen = ref.generator(M + N + K + E + seed)
    a = ref.randn(gen, M, K)
    shape = (K, N) if transposed else (N, K)
    w = ref.randn(gen, *((E,) if E else ()), *shape, scale=0.05)
    offsets = ref.cuts(M, E, kind) if E else None
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    got = zffn.bf16_matmul(a, w, offsets=offsets, transposed=transposed, y=y)
    assert got is y
    want, mag = ref.product(a, w, offsets, transposed)
    ref.check(y, want, ref.sum_bound(K) * mag, dtype)
    if E:
        assert torch.all(y[int(offsets[E]):] == 0)
    assert zffn.get_device_error() == zffn.OK


DENSE = [(1, 8, 8), (1, 2048, 1024), (3, 136, 264), (16, 1000, 72), (17, 256, 2048), (64, 384, 520), (65, 520, 136), (128, 256, 64),
         (129, 264, 1032), (257, 2056, 400), (700, 1032, 2056), (1500, 5136, 272), (3001, 128, 64)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K, dtype, transposed):
    run_product(M, N, K, 0, None, transposed, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (5, 7, 64), (40, 129, 136), (200, 515, 72), (1300, 2570, 136)])
def test_odd_columns(M, N, K, dtype):
    run_product(M, N, K, 0, None, False, dtype)
    run_product(M, N, K, 3, "borders", False, dtype)


GROUPED = [(1, 64, 64, 1), (8, 768, 256, 128), (37, 136, 1032, 5), (256, 264, 72, 100), (300, 1032, 264, 4096), (1860, 520, 136, 27),
           (1500, 1288, 272, 4), (4500, 648, 144, 3), (6000, 256, 64, 60), (2100, 2056, 520, 2)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K,E", GROUPED)
def test_grouped(M, N, K, E, kind, transposed):
    for dtype in DTYPES:
        run_product(M, N, K, E, kind, transposed, dtype)


GRADS = [(1, 8, 8, 0), (1, 264, 136, 0), (37, 136, 264, 0), (700, 392, 1032, 0), (4100, 128, 256, 0), (8, 768, 256, 16), (37, 136, 1032, 5),
         (256, 264, 72, 100), (300, 72, 264, 1000), (1860, 520, 136, 27), (1500, 1288, 272, 4), (5000, 136, 520, 3)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,E,kind", [(*g, k) for g in GRADS for k in (KINDS if g[3] else [None])])
def test_weights_gradient(M, N, K, E, kind, dtype):
    gen = ref.generator(M + N + K + E)
    dy, a = ref.randn(gen, M, N, scale=0.1), ref.randn(gen, M, K)
    offsets = ref.cuts(M, E, kind) if E else None
    dw = torch.full((E, N, K) if E else (N, K), 7.0, dtype=dtype, device="cuda")
    assert zffn.bf16_matmul_grad_w(dy, a, offsets=offsets, dw=dw) is dw
    want, tol = ref.grad_w(dy, a, offsets)
    ref.check(dw.view(want.shape), want, tol, dtype)
    assert zffn.get_device_error() == zffn.OK


def test_results_that_are_made():
    gen = ref.generator(1)
    a, w, dy = ref.randn(gen, 40, 64), ref.randn(gen, 3, 24, 64), ref.randn(gen, 40, 24)
    offsets = ref.cuts(40, 3, "unused")
    y = zffn.bf16_matmul(a, w, offsets)
    assert y.shape == (40, 24) and y.dtype == torch.bfloat16
    assert zffn.bf16_matmul(a, w, offsets, dtype=torch.float32).dtype == torch.float32
    dw = zffn.bf16_matmul_grad_w(dy, a, offsets)
    assert dw.shape == (3, 24, 64) and dw.dtype == torch.bfloat16
    assert zffn.bf16_matmul_grad_w(dy, a, dtype=torch.float32).shape == (24, 64)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,E,bad", [(70, 5, float("nan")), (400, 4, float("inf")), (1500, 4, float("nan"))])
def test_rows_of_others_do_not_matter(M, E, bad, transposed):
    # NaN and infinities in rows of no expert, of other experts, and in other experts' weights stay where they are
    gen = ref.generator(M)
    N, K = 264, 136
    a, dy = ref.randn(gen, M, K), ref.randn(gen, M, N)
    w = ref.randn(gen, E, *((K, N) if transposed else (N, K)))
    offsets = ref.cuts(M, E, "unused")
    cut = offsets.tolist()
    victim = max(range(E), key=lambda e: cut[e + 1] - cut[e])
    clean = zffn.bf16_matmul(a, w, offsets, transposed), zffn.bf16_matmul_grad_w(dy, a, offsets)
    a[cut[E]:], dy[cut[E]:] = bad, bad
    a[cut[victim]:cut[victim + 1]], dy[cut[victim]:cut[victim + 1]], w[victim] = bad, bad, bad
    y, dw = zffn.bf16_matmul(a, w, offsets, transposed), zffn.bf16_matmul_grad_w(dy, a, offsets)
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[cut[victim]:cut[victim + 1]] = False
    others = [e for e in range(E) if e != victim]
    assert torch.equal(y[rows], clean[0][rows]) and torch.equal(dw[others], clean[1][others])
    assert not torch.isfinite(y[~rows]).any() and not torch.isfinite(dw[victim]).any()


@pytest.mark.parametrize("M", [60, 1000])
def test_offsets_that_no_sort_writes(M):
    gen = ref.generator(2)
    E, N, K = 5, 136, 72
    a, w, dy = ref.randn(gen, M, K), ref.randn(gen, E, N, K), ref.randn(gen, M, N)
    for raw in ([0, M // 2, M // 4, M // 2, M, M], [-5, 3, 2, 40, 1 << 30, 7], [9, 20, 20, 10, 50, 50], [M, 0, 0, 0, 0, 0]):
        offsets = torch.tensor(raw, dtype=torch.int32, device="cuda")
        plain = torch.cummax(offsets.clamp(0, M), 0)[0].int()
        y = torch.full((M, N), 3.0, device="cuda")
        zffn.bf16_matmul(a, w, offsets, y=y)
        want, mag = ref.product(a, w, plain, False)
        first = int(plain[0])
        want[:first] = 3.0
        ref.check(y, want, ref.sum_bound(K) * mag)
        dw = zffn.bf16_matmul_grad_w(dy, a, offsets, dtype=torch.float32)
        ref.check(dw, *ref.grad_w(dy, a, plain))
    assert zffn.get_device_error() == zffn.OK


def test_unaligned_results_and_refusals():
    gen = ref.generator(3)
    a, w = ref.randn(gen, 300, 64), ref.randn(gen, 136, 64)
    want = zffn.bf16_matmul(a, w)
    flat = torch.zeros(300 * 136 + 1, dtype=torch.bfloat16, device="cuda")
    y = flat[1:].view(300, 136)
    zffn.bf16_matmul(a, w, y=y)
    assert torch.equal(y, want) and flat[0] == 0
    off = torch.zeros(300 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(300, 64)
    with pytest.raises(zffn.ZffnError):
        zffn.bf16_matmul(off, w)
    with pytest.raises(ValueError):
        zffn.bf16_matmul(a.t(), w)


def test_repeated_calls_are_equal():
    gen = ref.generator(4)
    for M, E in ((8, 8), (300, 20), (3000, 4)):
        a, w, dy = ref.randn(gen, M, 264), ref.randn(gen, E, 392, 264), ref.randn(gen, M, 392)
        offsets = ref.cuts(M, E, "random")
        y, dw = zffn.bf16_matmul(a, w, offsets, dtype=torch.float32), zffn.bf16_matmul_grad_w(dy, a, offsets, dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(zffn.bf16_matmul(a, w, offsets, dtype=torch.float32), y)
            assert torch.equal(zffn.bf16_matmul_grad_w(dy, a, offsets, dtype=torch.float32), dw)

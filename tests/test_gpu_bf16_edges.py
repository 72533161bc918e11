"""The bf16 products, SwiGLU and adapters at the ends of what their entry points allow: the widest and longest
operands, arrays of more than 2^31 elements, captured calls whose inputs change in place, chains of calls that are
not waited for, streams of another device, values whose products overflow.  Tolerances as in bf16_ref.py."""
import types

import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def adapters(gen, T, N, K, r, L):
    ids = torch.randint(-1, L, (T, 1), generator=gen, device="cuda").int()
    return (ids, ref.randn(gen, T, K), ref.randn(gen, T, N, scale=0.1), ref.randn(gen, L, r, K, scale=0.05), ref.randn(gen, L, N, r, scale=0.05),
            torch.rand((L,), generator=gen, device="cuda"), ref.randn(gen, T, N))


def adapter_step(ids, x, dy, A, B, scale, base):
    plan = zffn.moe_sort(ids, A.shape[0])
    out, v = zffn.lora_add(x, A, B, plan, scale=scale, base=base)
    return (out, v, *zffn.lora_grad(dy, x, v, A, B, plan, scale=scale))


@pytest.mark.parametrize("T", [5, 900])
def test_captured_adapters(T):
    N, K, r, L = 264, 520, 24, 6
    args = adapters(ref.generator(1), T, N, K, r, L)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        adapter_step(*args)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = adapter_step(*args)
    for seed in (2, 3):
        other = adapters(ref.generator(seed), T, N, K, r, L)
        want = adapter_step(*other)
        for a, b in zip(args, other):
            a.copy_(b)
        for _ in range(3):
            graph.replay()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("T", [5, 40, 900])
def test_chains_that_are_not_waited_for(T):
    # weights, scales and base change in place between calls that nothing waits for; each result goes to a copy
    N, K, r, L = 264, 520, 16, 40
    sets = [adapters(ref.generator(s), T, N, K, r, L) for s in range(4)]
    wants = []
    for s in sets:
        torch.cuda.synchronize()
        wants.append([t.clone() for t in adapter_step(*s)])
    now = [t.clone() for t in sets[0]]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        for t, s in zip(now, sets[i % 4]):
            t.copy_(s)
        got.append(adapter_step(*now))
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, wants[i % 4])), i
    # on top of each other: every call's base is the result before it
    ids, x, dy, A, B, scale, base = sets[0]
    plan = zffn.moe_sort(ids, L)
    a, b = base.clone(), base.clone()
    for _ in range(10):
        a, _ = zffn.lora_add(x, A, B, plan, base=a)
    for _ in range(10):
        zffn.lora_add(x, A, B, plan, base=b, out=b)
        torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_two_streams_of_adapters_and_products():
    jobs = [adapters(ref.generator(s), 600, 1032, 520, (16, 72, 128)[s], 5) for s in range(3)]
    wants = [adapter_step(*j) for j in jobs]
    w = ref.randn(ref.generator(9), 5, 1032, 520)
    cut = ref.cuts(600, 5, "even")
    products = [zffn.bf16_matmul(j[1], w, cut) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append((zffn.bf16_matmul(j[1], w, cut), adapter_step(*j), zffn.bf16_matmul(j[1], w, cut)))
        torch.cuda.synchronize()
        for g, want, y in zip(got, wants, products):
            assert torch.equal(g[0], y) and torch.equal(g[2], y)
            assert all(torch.equal(p, q) for p, q in zip(g[1], want))
    assert zffn.get_device_error() == zffn.OK


def test_stream_of_another_device_is_refused():
    here = torch.cuda.current_device()
    other = types.SimpleNamespace(cuda_stream=0, device_index=here + 1)      # (a stand-in: there is one device)
    x = torch.ones((4, 16), dtype=torch.bfloat16, device="cuda")
    A = torch.ones((1, 8, 16), dtype=torch.bfloat16, device="cuda")
    B = torch.ones((1, 16, 8), dtype=torch.bfloat16, device="cuda")
    plan = zffn.moe_sort(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 1)
    v = torch.ones((4, 8), device="cuda")
    for call in (lambda **kw: zffn.bf16_matmul(x, B[0].T.contiguous(), **kw), lambda **kw: zffn.bf16_matmul_grad_w(x, x, **kw),
                 lambda **kw: zffn.swiglu(x, **kw), lambda **kw: zffn.swiglu_grad(x[:, :8].contiguous(), x, **kw),
                 lambda **kw: zffn.lora_add(x, A, B, plan, **kw), lambda **kw: zffn.lora_grad(x, x, v, A, B, plan, **kw)):
        with pytest.raises(ValueError, match="stream must be on the current device"):
            call(stream=other)


def test_swiglu_where_products_would_overflow():
    # |g| up to where e^g is far below 1: the slopes are tiny, dh and u huge, the results in range
    g = torch.tensor([-80.0, -60.0, -1e20, 70.0, 1e20, -3.0], device="cuda")
    u = torch.tensor([1e30, -1e25, 1e30, 1e30, 1e10, 1e30], device="cuda")
    dh = torch.tensor([1e30, 1e25, 1e25, 1e5, 1e10, 1e5], device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        gu = torch.cat((g, u)).view(1, -1).to(dtype)
        g_, u_, d_ = gu[0, :6].double(), gu[0, 6:].double(), dh.to(dtype).double()
        s, rest = torch.sigmoid(g_), torch.sigmoid(-g_)
        want = torch.cat((d_ * (u_ * s * (1 + g_ * rest)), d_ * (g_ * s))).view(1, -1)
        got = zffn.swiglu_grad(dh.to(dtype).view(1, -1), gu).double()
        assert torch.isfinite(got).all()
        # 16 (1 + |g|) 2^-24 of the value as in test_gpu_swiglu.py, past |g| = 100 of exact zeros and ones; a bf16 result
        # is rounded by half a step more
        tol = 16 * (1 + torch.cat((g_, g_)).abs().clamp(max=100)) * ref.U32 * want.abs()
        tol = tol + (1.01 * ref.HALF_BF16 * want.abs() if dtype == torch.bfloat16 else 0) + 1e-37
        assert ((got - want).abs() <= tol).all(), (got, want)


@pytest.mark.parametrize("T,N,K,r,L", [(3, 8, 65536, 8, 2), (3, 65536, 8, 128, 2), (300, 8, 65536, 16, 3), (300, 65536, 8, 72, 3), (5000, 8, 8, 8, 4096)])
def test_widest_adapters(T, N, K, r, L):
    ids, x, dy, A, B, scale, base = adapters(ref.generator(T + r), T, N, K, r, L)
    plan = zffn.moe_sort(ids, L)
    want, tol, wv, vtol = ref.lora(x, A, B, plan, scale, base)
    out, v = zffn.lora_add(x, A, B, plan, scale=scale, base=base)
    ref.check(v, wv, vtol)
    ref.check(out, want, tol, torch.bfloat16)
    for g, (w, t) in zip(zffn.lora_grad(dy, x, v, A, B, plan, scale=scale, dtype=torch.float32), ref.lora_grad(dy, x, v, A, B, plan, scale, None)):
        ref.check(g, w, t)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("M,N,K,E", [(3, 65536, 8, 0), (300, 65536, 16, 0), (6000, 16, 8, 4096), (70000, 8, 16, 4096)])
def test_widest_products(M, N, K, E):
    gen = ref.generator(M + N)
    a, w = ref.randn(gen, M, K), ref.randn(gen, max(E, 1), N, K)
    cut = ref.cuts(M, E, "random") if E else None
    y = zffn.bf16_matmul(a, w if E else w[0], cut, dtype=torch.float32)
    want, mag = ref.product(a, w if E else w[0], cut, False)
    ref.check(y, want, ref.sum_bound(K) * mag)
    dy = ref.randn(gen, M, N)
    da = zffn.bf16_matmul(dy, w if E else w[0], cut, transposed=True, dtype=torch.float32)
    want, mag = ref.product(dy, w if E else w[0], cut, True)
    ref.check(da, want, ref.sum_bound(N) * mag)
    dw = zffn.bf16_matmul_grad_w(dy, a, cut, dtype=torch.float32)
    want, tol = ref.grad_w(dy, a, cut)
    ref.check(dw, want.view(dw.shape), tol.view(dw.shape))
    assert zffn.get_device_error() == zffn.OK


def some_rows(rows, cols):
    edge = 2 ** 31 // cols
    assert edge + 1 < rows - 2
    return torch.tensor([0, 1, edge - 1, edge, edge + 1, 2 * edge // 3, rows - 2, rows - 1], device="cuda")


@pytest.mark.parametrize("N,E,dtype", [(16400, 0, torch.bfloat16), (16401, 0, torch.float32), (16400, 4096, torch.bfloat16), (16400, 100, torch.float32)])
def test_far_results(N, E, dtype):
    # pairs, their stores by TMA and by the lanes; small tiles; pairs of experts
    K = 16
    M = 2 ** 31 // N + 500
    gen = ref.generator(N + E)
    a, w = ref.randn(gen, M, K), ref.randn(gen, max(E, 1), N, K, scale=0.1)
    cut = ref.cuts(M, E, "even") if E else None
    y = zffn.bf16_matmul(a, w if E else w[0], cut, dtype=dtype)
    at = some_rows(M, N)
    e = torch.searchsorted(cut, at.int(), right=True) - 1 if E else torch.zeros_like(at)
    x, ws = a[at].double(), w[e].double()
    want, mag = torch.einsum("rk,rnk->rn", x, ws), torch.einsum("rk,rnk->rn", x.abs(), ws.abs())
    ref.check(y[at], want, ref.sum_bound(K) * mag, dtype)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("transposed", [False, True])
def test_far_weights(transposed):
    E, N, K, M = 64, 8208, 4112, 12
    gen = ref.generator(3)
    w = torch.empty((E, K, N) if transposed else (E, N, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert w.numel() > 2 ** 31
    a = ref.randn(gen, M, K)
    cut = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    cut[E // 2:] = 5
    cut[E] = M
    y = zffn.bf16_matmul(a, w, cut, transposed, dtype=torch.float32)
    for e, rows in ((E // 2 - 1, slice(0, 5)), (E - 1, slice(5, M))):
        x, v = a[rows].double(), w[e].double() if transposed else w[e].double().T
        ref.check(y[rows], x @ v, ref.sum_bound(K) * (x.abs() @ v.abs()))
    if not transposed:
        dy = ref.randn(gen, M, N)
        del w
        dw = zffn.bf16_matmul_grad_w(dy, a, cut)
        for e, rows in ((0, slice(0, 0)), (E // 2 - 1, slice(0, 5)), (E - 1, slice(5, M))):
            d, x = dy[rows].double().T, a[rows].double()
            ref.check(dw[e], d @ x, ref.sum_bound(M) * (d.abs() @ x.abs()), torch.bfloat16)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("packed", [False, True])
def test_far_adapters(packed):
    N, K, r, L = 16400, 16, 8, 3
    T = 2 ** 31 // N + 300
    gen = ref.generator(5)
    ids = torch.randint(-1, L, (T, 1), generator=gen, device="cuda").int()
    if packed:
        ids = ids.sort(0)[0].contiguous()
    plan = zffn.moe_sort(ids, L)
    x, A, B = ref.randn(gen, T, K), ref.randn(gen, L, r, K), ref.randn(gen, L, N, r)
    base = torch.empty((T, N), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    at = some_rows(T, N)
    old = base[at].double()
    out, v = zffn.lora_add(x, A, B, plan, base=base)
    zffn.lora_add(x, A, B, plan, base=base, out=base)
    assert torch.equal(out[at], base[at])
    for i, t in enumerate(at.tolist()):
        e = int(ids[t])
        if e < 0:
            assert torch.equal(out[t].double(), old[i])
            continue
        vt, vm = x[t].double() @ A[e].double().T, x[t].double().abs() @ A[e].double().abs().T
        want, mag = old[i] + vt @ B[e].double().T, old[i].abs() + vm @ B[e].double().abs().T
        ref.check(out[t], want, (ref.sum_bound(K) + ref.sum_bound(3 * r)) * mag, torch.bfloat16)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("dtype,I", [(torch.bfloat16, 8192), (torch.float32, 8197)])
def test_far_swiglu(dtype, I):
    rows = 2 ** 31 // I + 100
    gen = ref.generator(I)
    gu = torch.empty((rows, 2 * I), dtype=dtype, device="cuda").normal_(generator=gen)
    at = some_rows(rows, I)
    h = zffn.swiglu(gu)
    assert torch.equal(h[at], zffn.swiglu(gu[at].contiguous()))
    some = gu[at].contiguous()
    zffn.swiglu_grad(h, gu, dgu=gu)
    assert torch.equal(gu[at], zffn.swiglu_grad(h[at].contiguous(), some))

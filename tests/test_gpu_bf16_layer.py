"""The bf16 operators together, as a program uses them: a routed layer's training step (sort, dispatch, gate and
up in one product, SwiGLU, down, combine, and the way back to tokens, routing weights and all weights), the same
step captured and replayed, adapters beside an 8-bit projection with their gradients, and other streams.

Tolerance of the chain: each step's bound (tests/bf16_ref.py) carried through the next by magnitudes."""
import pytest
import torch

from quantized_ffn_gb300 import zffn
from tests import bf16_ref as ref

pytestmark = pytest.mark.gpu


def layer(T, E, H, I, k, seed=0):
    gen = ref.generator(T + E + seed)
    x = ref.randn(gen, T, H)
    Wgu, Wd = ref.randn(gen, E, 2 * I, H, scale=0.05), ref.randn(gen, E, H, I, scale=0.05)
    ids = torch.randint(-1, E, (T, k), generator=gen, device="cuda").int()
    w = torch.rand((T, k), generator=gen, device="cuda")
    dy = torch.randn((T, H), generator=gen, device="cuda")
    return x, Wgu, Wd, ids, w, dy


def step(x, Wgu, Wd, ids, w, dy, E):
    plan = zffn.moe_sort(ids, E)
    xs = zffn.moe_dispatch(x, plan)
    gu = zffn.bf16_matmul(xs, Wgu, plan.offsets)
    h = zffn.swiglu(gu)
    rows = zffn.bf16_matmul(h, Wd, plan.offsets)
    y = zffn.moe_combine(rows, plan, w)
    drows, dw = zffn.moe_combine_grad(dy, rows, plan, w)
    dh = zffn.bf16_matmul(drows, Wd, plan.offsets, transposed=True)
    dWd = zffn.bf16_matmul_grad_w(drows, h, plan.offsets, dtype=torch.float32)
    dgu = zffn.swiglu_grad(dh, gu)
    dxs = zffn.bf16_matmul(dgu, Wgu, plan.offsets, transposed=True, dtype=torch.float32)
    dWgu = zffn.bf16_matmul_grad_w(dgu, xs, plan.offsets, dtype=torch.float32)
    return y, dw, zffn.moe_combine(dxs, plan), dWgu, dWd


def exact(x, Wgu, Wd, ids, w, dy, E):
    leaves = [t.double().requires_grad_() for t in (w, x, Wgu, Wd)]
    dw_, x_, gu_, d_ = leaves
    y = torch.zeros(dy.shape, dtype=torch.float64, device="cuda")
    for j in range(ids.shape[1]):
        for e in range(E):
            t = (ids[:, j] == e).nonzero().view(-1)
            g, u = (x_[t] @ gu_[e].T).chunk(2, 1)
            y = y.index_add(0, t, dw_[t, j, None] * ((torch.nn.functional.silu(g) * u) @ d_[e].T))
    grads = torch.autograd.grad(y, leaves, dy.double())
    return (y.detach(), *grads)


@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 136, 3), (64, 16, 1032, 512, 4), (600, 4, 520, 264, 2)])
def test_training_step(T, E, H, I, k):
    args = layer(T, E, H, I, k)
    got, want = step(*args, E), exact(*args, E)
    # a bf16 rounding at each of gu, h, rows, drows, dh, dgu: half a step of 2^-8 each, at most six in a chain, and
    # SwiGLU's slopes pass gu's on at most 1.1 (1 + |g|) times over; the roundings of a row are independent of each
    # other, so the whole is held to 8 half steps of its norm
    for g, x in zip(got, want):
        assert g.shape == x.shape
        assert (g.double() - x).norm() <= 8 * ref.HALF_BF16 * x.norm() + 1e-30
    assert zffn.get_device_error() == zffn.OK


def test_training_step_captured():
    T, E, H, I, k = 300, 8, 264, 136, 2
    args = layer(T, E, H, I, k)
    want = step(*args, E)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*args, E)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = step(*args, E)
    graph.replay()
    for g, x in zip(got, want):
        assert torch.equal(g, x)
    other = layer(T, E, H, I, k, seed=1)           # other routing and values in the same memory
    want = step(*other, E)
    for a, b in zip(args, other):
        a.copy_(b)
    for _ in range(3):
        graph.replay()
    for g, x in zip(got, want):
        assert torch.equal(g, x)
    assert zffn.get_device_error() == zffn.OK


@pytest.mark.parametrize("T", [1, 30, 400])
def test_adapters_beside_an_8_bit_projection(T):
    gen = ref.generator(T)
    N, K, r, L = 520, 1040, 16, 6
    q, s = zffn.fp8_quantize(ref.randn(gen, N, K, scale=0.05), block_rows=128)
    x, dy = ref.randn(gen, T, K), ref.randn(gen, T, N, scale=0.1)
    A, B = ref.randn(gen, L, r, K, scale=0.05), ref.randn(gen, L, N, r, scale=0.05)
    scale = torch.rand((L,), generator=gen, device="cuda")
    plan = zffn.moe_sort(torch.randint(-1, L, (T, 1), generator=gen, device="cuda").int(), L)
    xq, xs = zffn.fp8_quantize(x)
    y = zffn.fp8_matmul(xq, xs, q, s)
    want, tol, _, _ = ref.lora(x, A, B, plan, scale, y)
    out, v = zffn.lora_add(x, A, B, plan, scale, base=y, out=y)
    assert out is y
    ref.check(y, want, tol)
    # back: the frozen projection's share on the transposed bytes, the adapters' on top
    qt, st = q.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)[:, :512].contiguous(), s.t()[:, :4].contiguous()
    dq, ds = zffn.fp8_quantize(dy[:, :512].contiguous())
    base = zffn.fp8_matmul(dq, ds, qt, st)
    plain = ref.lora_grad(dy, x, v, A, B, plan, scale, base)
    got = zffn.lora_grad(dy, x, v, A, B, plan, scale, base=base, dx=base, dtype=torch.float32)
    for g, (w, t) in zip(got, plain):
        ref.check(g, w, t)
    assert zffn.get_device_error() == zffn.OK


def test_two_streams_at_once():
    # (no call shares a workspace, so calls on two streams may overlap)
    jobs = [layer(500, 8, 264, 136, 2, seed=i) for i in range(2)]
    want = [step(*j, 8) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(step(*j, 8))
        torch.cuda.synchronize()
        for g, x in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, x))


def test_results_on_a_given_stream():
    gen = ref.generator(7)
    a, w = ref.randn(gen, 2000, 1024), ref.randn(gen, 1024, 1024)
    want = zffn.bf16_matmul(a, w), zffn.bf16_matmul_grad_w(a, a), zffn.swiglu(a), zffn.swiglu_grad(a[:, :512].contiguous(), a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, run in enumerate((lambda **kw: zffn.bf16_matmul(a, w, **kw), lambda **kw: zffn.bf16_matmul_grad_w(a, a, **kw),
                             lambda **kw: zffn.swiglu(a, **kw), lambda **kw: zffn.swiglu_grad(h, a, **kw))):
        h = a[:, :512].contiguous()
        torch.cuda.synchronize()
        block = torch.empty_like(want[i])
        for _ in range(300):
            block.fill_(7)
        del block
        got = run(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want[i])

"""Plain 64-bit forms of the bf16 products, SwiGLU and the low-rank adapters (torch, on the inputs' device),
written from their definitions, each with the sum of magnitudes that rounding errors scale with."""
import numpy as np
import torch

U32 = 2.0 ** -24
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def sum_bound(terms):
    """What fp32 sums of `terms` bf16 products may be off by, as a part of the sum of magnitudes.  A product of
    two 8-bit significands is exact in fp32.  The tensor cores add 16 products at a time and may cut instead of
    round and align a group to its largest: 4 * 2^-24 for each group; and 32 more for joining partial sums (of
    at most 8 blocks, each rounded) and for the scale and base that are added at the end."""
    return (4 * (-(-terms // 16)) + 32) * U32


def check(got, want, tol, dtype=torch.float32):
    """got within tol of want; a bf16 result is rounded once more, by half a step at most."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    tol = tol + 1e-37
    if dtype == torch.bfloat16:
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * want.abs()
    bad = ~((got - want).abs() <= tol)
    at = bad.nonzero()[:5]
    assert not bad.any(), (int(bad.sum()), at.tolist(), got[bad][:5], want[bad][:5], tol[bad][:5])


def randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cuts(M, E, kind, seed=0):
    """Offsets of M rows over E groups: "even"; "random", many groups empty when E is large; "one": all in the
    middle one; "none": no row in any; "unused": rows past the last offset; "borders": at odd places."""
    rng = np.random.default_rng(seed + M + E)
    even = np.linspace(0, M, E + 1)
    if kind == "one":
        cut = np.zeros(E + 1)
        cut[E // 2 + 1:] = M
    elif kind == "none":
        cut = np.zeros(E + 1)
    elif kind == "unused":
        cut = np.sort(rng.integers(0, 2 * M // 3 + 1, E + 1))
        cut[0] = 0
    elif kind == "random":
        cut = np.sort(rng.integers(0, M + 1, E + 1))
        cut[0], cut[E] = 0, M
    elif kind == "borders":
        cut = np.clip(even + np.array([0] + [(37, -61, 5)[i % 3] for i in range(E - 1)] + [0]), 0, M)
        cut = np.maximum.accumulate(cut)
    else:
        cut = even
    return torch.from_numpy(cut.astype(np.int32)).cuda()


def groups(offsets, M):
    """(group, first row, past its last) of the groups that have rows."""
    at = [(0, M)] if offsets is None else zip(offsets[:-1].tolist(), offsets[1:].tolist())
    return [(e, lo, hi) for e, (lo, hi) in enumerate(at) if lo < hi]


def product(a, w, offsets, transposed):
    """(y, mag): rows of no group 0."""
    w = w if offsets is not None else w[None]
    N = w.shape[2] if transposed else w.shape[1]
    y = torch.zeros((a.shape[0], N), dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(y)
    for e, lo, hi in groups(offsets, a.shape[0]):
        x, v = a[lo:hi].double(), (w[e] if transposed else w[e].T).double()
        y[lo:hi], mag[lo:hi] = x @ v, x.abs() @ v.abs()
    return y, mag


def grad_w(dy, a, offsets):
    """(dw, tolerance of fp32 sums), [E, N, K]."""
    E = 1 if offsets is None else offsets.numel() - 1
    dw = torch.zeros((E, dy.shape[1], a.shape[1]), dtype=torch.float64, device=a.device)
    tol = torch.zeros_like(dw)
    for e, lo, hi in groups(offsets, a.shape[0]):
        d, x = dy[lo:hi].double().T, a[lo:hi].double()
        dw[e], tol[e] = d @ x, sum_bound(hi - lo) * (d.abs() @ x.abs())
    return dw, tol


def lora(x, A, B, plan, scale, base):
    """(out, its tolerance, v, its tolerance) of tokens sorted by adapter."""
    T, r, N = x.shape[0], A.shape[1], B.shape[1]
    out = torch.zeros((T, N), dtype=torch.float64, device=x.device) if base is None else base.double()
    tol = sum_bound(0) * out.abs()
    v = torch.zeros((T, r), dtype=torch.float64, device=x.device)
    vtol = torch.zeros_like(v)
    for e, lo, hi in groups(plan.offsets, T):
        t = plan.row_slot[lo:hi].long()
        s = 1.0 if scale is None else float(scale[e])
        a, b = A[e].double().T, B[e].double().T
        v[lo:hi] = s * (x[t].double() @ a)
        vtol[lo:hi] = sum_bound(x.shape[1]) * abs(s) * (x[t].double().abs() @ a.abs())
        out[t] += v[lo:hi] @ b
        tol[t] += vtol[lo:hi] @ b.abs() + sum_bound(3 * r) * ((v[lo:hi].abs() + vtol[lo:hi]) @ b.abs())
    return out, tol, v, vtol


def lora_grad(dy, x, v, A, B, plan, scale, base):
    """((dx, tol), (dA, tol), (dB, tol)); v is an input."""
    dx, dx_tol, dv, dv_tol = lora(dy, B.transpose(1, 2), A.transpose(1, 2), plan, scale, base)
    dA, dB = torch.zeros(A.shape, dtype=torch.float64, device=x.device), torch.zeros(B.shape, dtype=torch.float64, device=x.device)
    A_tol, B_tol = torch.zeros_like(dA), torch.zeros_like(dB)
    for e, lo, hi in groups(plan.offsets, x.shape[0]):
        t = plan.row_slot[lo:hi].long()
        xe, de, d, d_tol, ve = x[t].double(), dy[t].double(), dv[lo:hi], dv_tol[lo:hi], v[lo:hi].double()
        c = sum_bound(3 * (hi - lo))
        dA[e], dB[e] = d.T @ xe, de.T @ ve
        A_tol[e] = d_tol.T @ xe.abs() + c * ((d.abs() + d_tol).T @ xe.abs())
        B_tol[e] = c * (de.abs().T @ ve.abs())
    return (dx, dx_tol), (dA, A_tol), (dB, B_tol)

"""The expert training calls against plain 64-bit arithmetic.

Tolerances count roundings.  A bf16 result is off by at most half a step,
2^-8 of its value; an fp32 accumulation of n terms by at most n 2^-23 of the
sum of their absolute values (adds in the tensor cores may truncate); a hidden
value rounded to bf16 carries 2^-8 of its own absolute value into the sums it
enters.  Each bound is computed elementwise from the inputs.
"""
import math

import pytest
import torch

import mixture_experts_layer_54_b200 as moe

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def randn(*shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def table(sizes, aligned):
    """(offsets, rows or None, R, spans): packed groups after three rows of nobody
    and before two, or groups on multiples of 128 rows."""
    off, spans, at = [], [], 0 if aligned else 3
    for n in sizes:
        off.append(at)
        spans.append((at, at + n))
        at += -(-n // 128) * 128 if aligned else n
    return ints(off + [at]), ints(sizes) if aligned else None, at + 2, spans


def within(got, ref, bound, what=""):
    if ref.numel() == 0:
        return
    over = (got.to(F64) - ref).abs() - bound
    assert not torch.isnan(over).any(), what
    assert over.max().item() <= 0, (what, over.max().item(), int((over > 0).sum()))


SIZES = {
    "one_row": [1],
    "few_rows": [3, 0, 20, 33, 1, 32],
    "ragged": [0, 1, 127, 128, 129, 0, 300, 15, 16, 17],
    "long": [700, 513, 0, 1030],
    "single": [0, 0, 5],
    "empty": [0, 0],
}


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("N,K", [(64, 128), (264, 72), (8, 8), (328, 600)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_grouped_products(sizes, aligned, N, K, dtype):
    """Forward, input gradient and weight gradient; what lies outside the groups
    is NaN on the way in and a mark on the way out."""
    if dtype == F32:
        N, K = N - 1, K + 3
    off, rows, R, spans = table(SIZES[sizes], aligned)
    G = len(spans)
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    for lo, hi in spans:
        inside[lo:hi] = True
    x = randn(R, K, seed=1, dtype=dtype)
    dy = randn(R, N, seed=2, dtype=dtype)
    x[~inside] = float("nan")
    dy[~inside] = float("nan")
    W = randn(G, N, K, seed=3, dtype=dtype, scale=K ** -0.5)
    mark = 7.0
    y = torch.full((R, N), mark, dtype=dtype, device="cuda")
    dx = torch.full((R, K), mark, dtype=dtype, device="cuda")
    ws = moe.workspace(moe.lib().moe_grouped_workspace_size(int(dtype == BF), G, R, N, K), "cuda")
    ws.fill_(255)   # whatever the workspace held must not show
    moe.moe_grouped_matmul(x, W, off, rows, y=y, ws=ws)
    assert moe.moe_device_status(ws) == 0
    moe.moe_grouped_matmul_dx(dy, W, off, rows, dx=dx, ws=ws)
    assert moe.moe_device_status(ws) == 0
    dW = moe.moe_grouped_matmul_dw(dy, x, off, rows, ws=ws)
    dW32 = moe.moe_grouped_matmul_dw(dy, x, off, rows, out_dtype=F32, ws=ws)
    add = randn(G, N, K, seed=4, dtype=dtype)
    dWa = moe.moe_grouped_matmul_dw(dy, x, off, rows, add=add, ws=ws)
    acc = dW32.clone()
    moe.moe_grouped_matmul_dw(dy, x, off, rows, add=acc, dW=acc, ws=ws)
    assert moe.moe_device_status(ws) == 0
    assert (y[~inside] == mark).all() and (dx[~inside] == mark).all()
    h = HALF[dtype]
    for g, (lo, hi) in enumerate(spans):
        a, b, w = x[lo:hi].to(F64), dy[lo:hi].to(F64), W[g].to(F64)
        n = hi - lo
        r = a @ w.T
        within(y[lo:hi], r, h * r.abs() + K * 2.0 ** -23 * (a.abs() @ w.abs().T), "y")
        r = b @ w
        within(dx[lo:hi], r, h * r.abs() + N * 2.0 ** -23 * (b.abs() @ w.abs()), "dx")
        r, s = b.T @ a, (n + 1) * 2.0 ** -23 * (b.abs().T @ a.abs())
        within(dW[g], r, h * r.abs() + s, "dW")
        within(dW32[g], r, 2.0 ** -24 * r.abs() + s, "dW fp32")
        r2 = r + add[g].to(F64)
        s2 = s + 2.0 ** -23 * (r2.abs() + add[g].to(F64).abs())
        within(dWa[g], r2, h * r2.abs() + s2, "dW added")
        within(acc[g], 2 * r, 2.0 ** -22 * r.abs() + 2 * s, "dW accumulated")


@pytest.mark.parametrize("sizes,N,K", [([600], 256, 4096), ([5, 40], 136, 8192), ([30, 700], 72, 5000),
                                       ([9000, 3, 0, 2000], 128, 128), ([3000], 320, 264),
                                       ([20, 17, 9, 31, 2], 264, 3000)])
def test_long_contractions_are_cut_and_joined(sizes, N, K):
    """Few tiles over long contractions: parts of a tile run side by side.  Every
    run gives the same bits, whichever part is last and whatever the workspace
    held."""
    off, rows, R, spans = table(sizes, False)
    G = len(spans)
    x, dy = randn(R, K, seed=1), randn(R, N, seed=2)
    W = randn(G, N, K, seed=3, scale=K ** -0.5)
    ws = moe.workspace(moe.lib().moe_grouped_workspace_size(1, G, R, N, K), "cuda")
    results = []
    for fill in (255, 0, 7):
        ws.fill_(fill)
        for _ in range(3):
            results.append((moe.moe_grouped_matmul(x, W, off, y=torch.zeros_like(dy), ws=ws),
                            moe.moe_grouped_matmul_dx(dy, W, off, dx=torch.zeros_like(x), ws=ws),
                            moe.moe_grouped_matmul_dw(dy, x, off, out_dtype=F32, ws=ws)))
            assert moe.moe_device_status(ws) == 0
    for r in results[1:]:
        for a, b in zip(r, results[0]):
            assert torch.equal(a, b)
    y, dx, dW = results[0]
    for g, (lo, hi) in enumerate(spans):
        a, b, w = x[lo:hi].to(F64), dy[lo:hi].to(F64), W[g].to(F64)
        r = a @ w.T
        within(y[lo:hi], r, 2.0 ** -8 * r.abs() + K * 2.0 ** -23 * (a.abs() @ w.abs().T), "y")
        r = b @ w
        within(dx[lo:hi], r, 2.0 ** -8 * r.abs() + N * 2.0 ** -23 * (b.abs() @ w.abs()), "dx")
        r = b.T @ a
        # summed in accumulators of 512 rows: the truncations do not add up over all of them
        n = min(hi - lo, 512) + (hi - lo) / 512 + 20
        within(dW[g], r, 2.0 ** -24 * r.abs() + n * 2.0 ** -23 * (b.abs().T @ a.abs()), "dW")


def test_calls_side_by_side_on_two_streams():
    """Two products on two streams with workspaces of their own give the bits of
    the same calls in turn."""
    off, _, R, spans = table([600, 40, 300], False)
    W = randn(3, 264, 2048, seed=3, scale=1 / 45)
    xs = [randn(R, 2048, seed=s) for s in (1, 2)]
    want = [moe.moe_grouped_matmul(x, W, off, y=torch.zeros((R, 264), dtype=BF, device="cuda"))
            for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                y = torch.zeros((R, 264), dtype=BF, device="cuda")
                got.append(moe.moe_grouped_matmul(x, W, off, y=y))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_grouped_products_of_no_rows():
    off = ints([0, 0, 0])
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    W = randn(2, 32, 64, seed=1)
    assert moe.moe_grouped_matmul(x, W, off).shape == (0, 32)
    dy = torch.empty((0, 32), dtype=BF, device="cuda")
    assert moe.moe_grouped_matmul_dx(dy, W, off).shape == (0, 64)
    for dtype in (BF, F32):
        dW = moe.moe_grouped_matmul_dw(dy, x, off, out_dtype=dtype)
        assert (dW == 0).all()
    add = randn(2, 32, 64, seed=2)
    assert torch.equal(moe.moe_grouped_matmul_dw(dy, x, off, add=add), add)


def test_tables_outside_the_buffers_are_held_inside():
    """Entries below 0, past R or decreasing: no access outside, the rows that the
    held table leaves to a group are its own."""
    R, N, K = 200, 64, 64
    x, W = randn(R, K, seed=1), randn(3, N, K, seed=2, scale=1 / 8)
    y = torch.full((R, N), 3.0, dtype=BF, device="cuda")
    moe.moe_grouped_matmul(x, W, ints([-50, 100, 90, 1 << 30]), ints([1 << 30, 5, 60]), y=y)
    for g, (lo, hi) in enumerate([(0, 100), (0, 0), (90, 150)]):
        if g == 2:
            lo = 100   # rows 90..99 belong to two groups: either value is right
        r = x[lo:hi].to(F64) @ W[g].to(F64).T
        if g == 0:
            r, lo, hi = r[:90], 0, 90
        within(y[lo:hi], r, 2.0 ** -8 * r.abs() + K * 2.0 ** -23 *
               (x[lo:hi].to(F64).abs() @ W[g].to(F64).abs().T))
    assert (y[150:] == 3.0).all()


def ffn_reference(x, dy, W1, W3, W2, act):
    """((gradients), (bounds)) of one expert in 64 bits; the bounds carry the
    roundings of h, du and dv and of the accumulations."""
    x, dy, W1, W2 = (t.to(F64) for t in (x, dy, W1, W2))
    d, n = x.shape[1], x.shape[0]
    F = W1.shape[0]
    e23, h8 = 2.0 ** -23, 2.0 ** -8
    u, dh = x @ W1.T, dy @ W2
    eu = d * e23 * (x.abs() @ W1.abs().T) + 2.0 ** -20 * u.abs()
    edh = d * e23 * (dy.abs() @ W2.abs())
    if act == 0:
        cdf = 0.5 * (1 + torch.erf(u / math.sqrt(2)))
        slope = cdf + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
        h, du = u * cdf, dh * slope
        # |gelu'| <= 1.13, |gelu''| <= 0.8; fast exponential: 2^-20
        eh = h8 * h.abs() + 1.13 * eu
        edu = h8 * du.abs() + 1.13 * edh + (0.8 * eu + 2.0 ** -20) * dh.abs()
        dv = None
    else:
        W3 = W3.to(F64)
        v = x @ W3.T
        ev = d * e23 * (x.abs() @ W3.abs().T)
        s = torch.sigmoid(u)
        silu, slope = u * s, s + u * s * (1 - s)
        h, du, dv = silu * v, dh * v * slope, dh * silu
        # |silu'| <= 1.1, |silu''| <= 0.5; fast exponential and division: 2^-20
        eh = h8 * h.abs() + 1.1 * eu * v.abs() + silu.abs() * ev
        edv = h8 * dv.abs() + silu.abs() * edh + 1.1 * eu * dh.abs()
        edu = (h8 * du.abs() + 1.1 * (v.abs() * edh + dh.abs() * ev) +
               (0.5 * eu + 2.0 ** -20 * (1 + u.abs())) * (dh * v).abs())
    out = lambda r, e: h8 * r.abs() + (1 + h8) * e
    dx = du @ W1
    bx = edu @ W1.abs() + 2 * F * e23 * (du.abs() @ W1.abs())
    if act:
        dx = dx + dv @ W3
        bx = bx + edv @ W3.abs() + 2 * F * e23 * (dv.abs() @ W3.abs())
    acc = n * e23
    g1, b1 = du.T @ x, edu.T @ x.abs() + acc * (du.abs().T @ x.abs())
    g2, b2 = dy.T @ h, dy.abs().T @ eh + acc * (dy.abs().T @ h.abs())
    g3 = b3 = None
    if act:
        g3, b3 = dv.T @ x, edv.T @ x.abs() + acc * (dv.abs().T @ x.abs())
    return (dx, g1, g3, g2), (out(dx, bx), out(g1, b1), None if g3 is None else out(g3, b3),
                              out(g2, b2)), bx


def ffn_case(T, d, E, k, F, act, S=0, Fs=0, dtype=1, sizes=None, seed=0):
    cfg = moe.moe_config(T=T, d=d, E=E, k=k, d_ff=F, act=act, dtype=dtype, cf=math.inf,
                         n_shared=S, d_ff_shared=Fs)
    R = moe.moe_perm_rows(cfg)
    dt = BF if dtype else F32
    off, kept, used, spans = table(sizes, True)
    x = randn(R, d, seed=seed + 1, dtype=dt)
    dY = randn(R, d, seed=seed + 2, dtype=dt)
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    for lo, hi in spans:
        inside[lo:hi] = True
    x[~inside] = float("nan")
    dY[~inside] = float("nan")
    W = [randn(E, F, d, seed=seed + 3, dtype=dt, scale=d ** -0.5),
         randn(E, F, d, seed=seed + 4, dtype=dt, scale=d ** -0.5) if act else None,
         randn(E, d, F, seed=seed + 5, dtype=dt, scale=F ** -0.5)]
    sh = {}
    if S:
        sh = dict(x=randn(T, d, seed=seed + 6, dtype=dt), dY_shared=randn(T, d, seed=seed + 7, dtype=dt),
                  Ws1=randn(S, Fs, d, seed=seed + 8, dtype=dt, scale=d ** -0.5),
                  Ws3=randn(S, Fs, d, seed=seed + 9, dtype=dt, scale=d ** -0.5) if act else None,
                  Ws2=randn(S, d, Fs, seed=seed + 10, dtype=dt, scale=Fs ** -0.5))
    return cfg, x, off, kept, dY, W, sh, spans, inside


FFN_CASES = {
    # act, sizes (sum <= T k), S, Fs, d, F
    "gelu_small": (0, [0, 1, 130, 60], 0, 0, 128, 64),
    "swiglu_small": (1, [17, 0, 128, 96], 0, 0, 64, 192),
    "gelu_pair": (0, [700, 513, 400, 1], 1, 64, 192, 320),
    "swiglu_pair": (1, [129, 800, 0, 650], 2, 192, 320, 128),
    "swiglu_one_token": (1, [1, 0, 0, 0], 3, 64, 64, 64),
    # long contractions beside a shared expert of one block: parts of cut tiles stay empty
    "swiglu_long_beside_short": (1, [90, 70, 40, 33], 1, 64, 64, 2048),
    "gelu_long_beside_short": (0, [90, 70, 40, 33], 1, 64, 64, 4096),
}


@pytest.mark.parametrize("name", list(FFN_CASES))
@pytest.mark.parametrize("dtype", [1, 0])
def test_ffn_backward(name, dtype):
    act, sizes, S, Fs, d, F = FFN_CASES[name]
    T = sum(sizes)
    cfg, x, off, kept, dY, W, sh, spans, inside = ffn_case(T, d, 4, 1, F, act, S, Fs, dtype, sizes)
    dx = torch.full_like(x, 7.0)
    ws = moe.workspace(moe.moe_ffn_backward_workspace_size(cfg), "cuda")
    ws.fill_(255)   # whatever the workspace held must not show
    g = moe.moe_expert_ffn_backward(cfg, x, off, kept, dY, *W, **sh, dx_perm=dx, ws=ws)
    assert moe.moe_device_status(ws) == 0
    assert (dx[~inside] == 7.0).all()
    acc = moe.FFNGrads(**{k: None if v is None else (v.float().clone() if k.startswith("dW") else v.clone())
                          for k, v in vars(g).items()})
    first = {k: v.clone() for k, v in vars(acc).items() if v is not None}
    moe.moe_expert_ffn_backward(cfg, x, off, kept, dY, *W, **sh, grads=acc, accumulate=True, ws=ws)
    for e, (lo, hi) in enumerate(spans):
        W3 = W[1][e] if act else None
        ref, bound, _ = ffn_reference(x[lo:hi], dY[lo:hi], W[0][e], W3, W[2][e], act)
        got = (dx[lo:hi], g.dW1[e], g.dW3[e] if act else None, g.dW2[e])
        for what, a, r, b in zip(("dx", "dW1", "dW3", "dW2"), got, ref, bound):
            if r is not None:
                within(a, r, b, f"{what}[{e}]")
                if what != "dx":   # what was there, plus the gradient again
                    base = first[what][e].to(F64)
                    within(getattr(acc, what)[e], base + r, b + 2.0 ** -23 * (base + r).abs())
    if S:
        dxs, bxs = 0, 0
        for s in range(S):
            ref, bound, bx = ffn_reference(sh["x"], sh["dY_shared"], sh["Ws1"][s],
                                           sh["Ws3"][s] if act else None, sh["Ws2"][s], act)
            dxs, bxs = dxs + ref[0], bxs + S * bx
            for what, a, r, b in zip(("dWs1", "dWs3", "dWs2"), (g.dWs1, g.dWs3, g.dWs2), ref[1:],
                                     bound[1:]):
                if r is not None:
                    within(a[s], r, b, f"{what}[{s}]")
        within(g.dx_shared, dxs, 2.0 ** -8 * dxs.abs() + (1 + 2.0 ** -8) * bxs, "dx_shared")


def test_ffn_backward_of_no_tokens():
    cfg = moe.moe_config(T=0, d=64, E=2, k=1, d_ff=64, act=1, dtype=1, cf=1.0, n_shared=1,
                         d_ff_shared=64)
    R = moe.moe_perm_rows(cfg)
    x = torch.full((R, 64), float("nan"), dtype=BF, device="cuda")
    W = [randn(2, 64, 64, seed=i) for i in range(3)]
    Ws = [randn(1, 64, 64, seed=i) for i in range(3)]
    none = torch.empty((0, 64), dtype=BF, device="cuda")
    g = moe.moe_expert_ffn_backward(cfg, x, ints([0, 0, 0]), ints([0, 0]), x, *W, x=none,
                                    dY_shared=none, Ws1=Ws[0], Ws3=Ws[1], Ws2=Ws[2])
    for t in (g.dW1, g.dW3, g.dW2, g.dWs1, g.dWs3, g.dWs2):
        assert (t == 0).all()


@pytest.mark.parametrize("T,d,E,k,cf,dtype", [(1, 64, 2, 1, 1.0, 1), (33, 64, 4, 2, 1.0, 1),
                                              (300, 1024, 16, 6, 1.0, 1), (257, 2112, 9, 8, 1.2, 1),
                                              (64, 36, 4, 3, 1.0, 0), (50, 1540, 5, 5, 1.5, 0)])
def test_combine_backward(T, d, E, k, cf, dtype):
    dt = BF if dtype else F32
    cfg = moe.moe_config(T=T, d=d, E=E, k=k, d_ff=64, act=1, dtype=dtype, cf=cf)
    topk = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k]
                        for t in range(T)]).int().cuda()
    cap = moe.moe_capacity(cfg, topk)
    R = moe.moe_perm_rows(cfg)
    gates = randn(T, k, seed=3, dtype=F32)
    gates[::7, 0] = 0.0
    dy, Y = randn(T, d, seed=1, dtype=dt), randn(R, d, seed=2, dtype=dt)
    row = cap.offsets.long()[topk.long()] + cap.pos.long()
    keep = cap.keep.bool()
    taken = torch.zeros(R, dtype=torch.bool, device="cuda")
    taken[row[keep]] = True
    Y[~taken] = float("nan")
    dY = torch.full((R, d), 7.0, dtype=dt, device="cuda")
    _, dg = moe.moe_combine_backward(cfg, dy, Y, gates, topk, cap.pos, cap.keep, cap.offsets,
                                     dY_perm=dY)
    assert (dY[~taken] == 7.0).all()
    assert (dg[~keep] == 0).all()
    t, j = torch.nonzero(keep, as_tuple=True)
    g64, dy64 = gates[t, j].to(F64)[:, None], dy[t].to(F64)
    ref = g64 * dy64
    # one fp32 product, one rounding
    within(dY[row[t, j]], ref, (HALF[dt] + 2.0 ** -24) * ref.abs() * 1.01)
    y64 = Y[row[t, j]].to(F64)
    within(dg[t, j], (dy64 * y64).sum(1), (d + 8) * 2.0 ** -24 * (dy64 * y64).abs().sum(1))


def newton_schulz(G, steps, coeffs, eps=1e-7):
    a, b, c = coeffs
    X = G.to(F64)
    X = X / (torch.linalg.matrix_norm(X)[..., None, None] + eps)
    for _ in range(steps):
        if X.shape[-2] <= X.shape[-1]:
            A = X @ X.mT
            X = a * X + (b * A + c * A @ A) @ X
        else:
            A = X.mT @ X
            X = a * X + X @ (b * A + c * A @ A)
    return X


QUINTIC = (3.4445, -4.7750, 2.0315)
# rounding to bf16 (2^-8) and the last step's fp16 operands: X, A and B are each
# off by 2^-11, and enter with factors below 3.5, 9 and 3
NS_TOL = 2.0 ** -8 + 16 * 2.0 ** -11


@pytest.mark.parametrize("E,m,n", [(1, 1, 1), (2, 1, 40), (3, 37, 51), (2, 51, 37), (4, 64, 32),
                                   (2, 300, 700), (3, 520, 264), (1, 256, 1000), (1, 130, 4100),
                                   (2, 129, 129), (5, 16, 16),
                                   (1, 128, 320), (2, 320, 128), (1, 128, 321), (200, 24, 72)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["noise", "low_rank"])
def test_orthogonalize(E, m, n, dtype, kind):
    G = randn(E, m, n, seed=m + n, dtype=F32, scale=1e-3)
    if kind == "low_rank":
        r = min(m, n, 4)
        u, v = randn(E, m, r, seed=1, dtype=F32), randn(E, r, n, seed=2, dtype=F32)
        G = u @ v + 10 * G
    G = G.to(dtype)
    ws = moe.workspace(moe.moe_orthogonalize_workspace_size(E, m, n, 5), "cuda")
    ws.fill_(255)
    U = moe.moe_orthogonalize(G, ws=ws)
    assert moe.moe_device_status(ws) == 0
    ref = newton_schulz(G, 5, QUINTIC)
    for e in range(E):
        rel = ((U[e].to(F64) - ref[e]).norm() / ref[e].norm()).item()
        assert rel <= NS_TOL, (e, rel)


@pytest.mark.parametrize("steps,coeffs,scale", [(1, QUINTIC, 1.0), (2, QUINTIC, 0.5),
                                                (8, (1.5, -0.5, 0.0), 0.2), (3, (2.0, -1.5, 0.5), 1.0)])
def test_orthogonalize_steps_and_coefficients(steps, coeffs, scale):
    for m, n in ((96, 160), (160, 96)):
        G = randn(2, m, n, seed=5, dtype=F32)
        U = moe.moe_orthogonalize(G, steps=steps, coeffs=coeffs, scale=scale)
        ref = scale * newton_schulz(G, steps, coeffs)
        assert ((U.to(F64) - ref).norm() / ref.norm()).item() <= NS_TOL


def test_orthogonalize_zeros_infinities_and_one_matrix():
    G = randn(4, 48, 40, seed=1)
    G[1] = 0
    G[2, 3, 4] = float("inf")
    U = moe.moe_orthogonalize(G)
    assert (U[1] == 0).all() and torch.isnan(U[2]).all()
    ref = newton_schulz(G, 5, QUINTIC)
    for e in (0, 3):
        assert ((U[e].to(F64) - ref[e]).norm() / ref[e].norm()).item() <= NS_TOL
    # one matrix, and an input and an output off the 16-byte grid
    flat, out = torch.zeros(48 * 40 + 1, dtype=BF, device="cuda"), torch.zeros(
        48 * 40 + 1, dtype=BF, device="cuda")
    flat[1:] = G[0].reshape(-1)
    one = moe.moe_orthogonalize(flat[1:].view(48, 40), U=out[1:].view(48, 40))
    assert torch.equal(one, U[0])


@pytest.mark.parametrize("scale", [1e-12, 1e10])
def test_orthogonalize_of_far_magnitudes(scale):
    """The norm decides the scale: with eps 0 a small or large update gives what
    the same update near 1 gives."""
    G = randn(1, 64, 96, seed=3, dtype=F32)
    want = moe.moe_orthogonalize(G, eps=0.0).to(F64)
    got = moe.moe_orthogonalize(G * scale, eps=0.0).to(F64)
    assert ((got - want).norm() / want.norm()).item() <= 2 * NS_TOL


def layer(T=200, d=128, E=4, k=2, F=192, act=1, S=1, Fs=64):
    cfg = moe.moe_config(T=T, d=d, E=E, k=k, d_ff=F, act=act, dtype=1, cf=1.0, n_shared=S,
                         d_ff_shared=Fs)
    w = dict(W1=randn(E, F, d, seed=11, scale=d ** -0.5), W3=randn(E, F, d, seed=12, scale=d ** -0.5),
             W2=randn(E, d, F, seed=13, scale=F ** -0.5), Ws1=randn(S, Fs, d, seed=14, scale=d ** -0.5),
             Ws3=randn(S, Fs, d, seed=15, scale=d ** -0.5), Ws2=randn(S, d, Fs, seed=16, scale=Fs ** -0.5))
    return cfg, w, randn(T, d, seed=17), randn(d, E, seed=18, dtype=F32, scale=d ** -0.5)


def step(cfg, w, x, W_r, dy):
    """One training step of the experts through the public calls."""
    topk, gates, _, _, _ = moe.moe_route(cfg, x, W_r)
    cap = moe.moe_capacity(cfg, topk)
    xp = moe.moe_dispatch(cfg, x, topk, cap.pos, cap.keep, cap.offsets)
    Yp, Ys, _ = moe.moe_expert_ffn(cfg, xp, cap.offsets, w["W1"], w["W3"], w["W2"], x=x,
                                   Ws1=w["Ws1"], Ws3=w["Ws3"], Ws2=w["Ws2"])
    y = moe.moe_combine(cfg, Yp, Ys, gates, topk, cap.pos, cap.keep, cap.offsets)
    dYp, dgates = moe.moe_combine_backward(cfg, dy, Yp, gates, topk, cap.pos, cap.keep, cap.offsets)
    g = moe.moe_expert_ffn_backward(cfg, xp, cap.offsets, cap.kept, dYp, w["W1"], w["W3"], w["W2"],
                                    x=x, dY_shared=dy, Ws1=w["Ws1"], Ws3=w["Ws3"], Ws2=w["Ws2"])
    dx = moe.moe_combine(cfg, g.dx_perm, g.dx_shared, torch.ones_like(gates), topk, cap.pos,
                         cap.keep, cap.offsets)
    U = [moe.moe_orthogonalize(t) for t in (g.dW1, g.dW3, g.dW2)]
    return y, dx, dgates, g, U, (topk, gates, cap)


def autograd_layer(cfg, w, x, gates, topk, keep, act):
    """The layer in 64-bit torch with autograd, routing given."""
    y = torch.zeros_like(x)
    ffn = lambda v, a, b, c: (torch.nn.functional.silu(v @ a.T) * (v @ b.T)) @ c.T
    for e in range(cfg.E):
        for j in range(cfg.k):
            t = torch.nonzero((topk[:, j] == e) & keep[:, j].bool())[:, 0]
            if t.numel():
                y = y.index_add(0, t, gates[t, j, None] * ffn(x[t], w["W1"][e], w["W3"][e], w["W2"][e]))
    for s in range(cfg.n_shared):
        y = y + ffn(x, w["Ws1"][s], w["Ws3"][s], w["Ws2"][s])
    return y


def test_training_step_matches_autograd_in_64_bits():
    """The calls in a row are the layer's gradient: against autograd, and against
    a difference quotient along a random direction."""
    cfg, w, x, W_r = layer()
    dy = randn(cfg.T, cfg.d, seed=20)
    y, dx, dgates, g, U, (topk, gates, cap) = step(cfg, w, x, W_r, dy)
    w64 = {n: t.to(F64).requires_grad_() for n, t in w.items()}
    x64, g64 = x.to(F64).requires_grad_(), gates.to(F64).requires_grad_()
    y64 = autograd_layer(cfg, w64, x64, g64, topk, cap.keep, cfg.act)
    y64.backward(dy.to(F64))
    # a chain of at most six bf16 roundings (x_perm is exact): Y, dY, h, du or dv,
    # dx of a slot, the result; in 2-norm each adds at most 2^-8, sums of signed
    # terms at most a factor 2 on top
    tol = 12 * 2.0 ** -8
    rel = lambda a, b: ((a.to(F64) - b).norm() / b.norm()).item()
    assert rel(y, y64.detach()) <= tol
    assert rel(dx, x64.grad) <= tol
    assert rel(dgates * cap.keep, g64.grad) <= tol
    for name in ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2"):
        assert rel(getattr(g, "d" + name), w64[name].grad) <= tol, name
    dirs = {n: torch.randn_like(t) for n, t in w64.items()}
    loss = lambda s: (autograd_layer(cfg, {n: t.detach() + s * dirs[n] for n, t in w64.items()},
                                     x64.detach(), g64.detach(), topk, cap.keep, cfg.act) *
                      dy.to(F64)).sum()
    slope = ((loss(1e-5) - loss(-1e-5)) / 2e-5).item()
    ours = sum((getattr(g, "d" + n).to(F64) * dirs[n]).sum().item() for n in dirs)
    size = math.sqrt(sum((t.grad.norm().item() * dirs[n].norm().item() / math.sqrt(dirs[n].numel())) ** 2
                         for n, t in w64.items()))
    assert abs(ours - slope) <= 6 * tol * size   # a projection of the error: six of its deviations
    for u, t in zip(U, (g.dW1, g.dW3, g.dW2)):
        ref = newton_schulz(t, 5, QUINTIC)
        assert rel(u, ref) <= NS_TOL


def test_training_step_captured_and_replayed():
    """Two steps captured in two graphs give, replayed in turn on new inputs, the
    bits of the eager calls; a second stream beside them changes nothing."""
    cfg, w, x, W_r = layer()
    dy = randn(cfg.T, cfg.d, seed=20)
    step(cfg, w, x, W_r, dy)
    xs, dys = x.clone(), dy.clone()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, dx, dgates, g, U, _ = step(cfg, w, xs, W_r, dys)
        graphs.append(gr)
        outs.append((y, dx, dgates, g.dW1, g.dW3, g.dW2, g.dWs1, g.dWs3, g.dWs2, *U))
    for i in range(3):
        xs.copy_(randn(cfg.T, cfg.d, seed=30 + i))
        dys.copy_(randn(cfg.T, cfg.d, seed=40 + i))
        y, dx, dgates, g, U, _ = step(cfg, w, xs, W_r, dys)
        want = [t.clone() for t in (y, dx, dgates, g.dW1, g.dW3, g.dW2, g.dWs1, g.dWs3, g.dWs2, *U)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step(cfg, w, xs, W_r, dys)
        for gr, out in zip(graphs, outs):
            for t in out:
                t.zero_()
            gr.replay()
            for a, b in zip(out, want):
                assert torch.equal(a, b)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other[1], want[1])


@pytest.mark.parametrize("G,N,K", [(7, 2048, 17280), (1, 14336, 24576)])
def test_parts_of_few_row_tiles_stay_inside_the_workspace(G, N, K):
    """Around a hundred tiles of 32 rows over a long contraction are cut into more
    parts than tiles of 128 rows could be: nothing is written behind the
    workspace, and the rows are right."""
    R = 5 * G
    off = ints([5 * g for g in range(G + 1)])
    x = randn(R, K, seed=1)
    W = randn(G, N, K, seed=3, scale=K ** -0.5)
    need = moe.lib().moe_grouped_workspace_size(1, G, R, N, K)
    buf = moe.workspace(need + (96 << 20), "cuda")
    buf.fill_(165)
    y = moe.moe_grouped_matmul(x, W, off, ws=buf[:need])
    assert moe.moe_device_status(buf[:need]) == 0
    assert (buf[need:] == 165).all()
    for g in range(G):
        a, w = x[5 * g:5 * g + 5].to(F64), W[g].to(F64)
        r = a @ w.T
        within(y[5 * g:5 * g + 5], r, 2.0 ** -8 * r.abs() + K * 2.0 ** -23 * (a.abs() @ w.abs().T))


@pytest.mark.parametrize("m,n", [(48, 80), (300, 700)])
@pytest.mark.parametrize("power", [-130, -90, 90, 110])
def test_orthogonalize_of_squares_outside_fp32(m, n, power):
    """Elements whose squares overflow or vanish in fp32: a power of two changes
    nothing with eps 0.  (2^-130 elements are denormal: rounded to 2^-149, so to
    2^-19 of the largest at least.)"""
    G = randn(2, m, n, seed=3, dtype=F32)
    G[1] = 0
    G[1, 0, 0] = 1.0   # one element
    got = moe.moe_orthogonalize(G * 2.0 ** power, eps=0.0).to(F64)
    ref = newton_schulz(G, 5, QUINTIC, eps=0.0)
    for e in range(2):
        assert ((got[e] - ref[e]).norm() / ref[e].norm()).item() <= NS_TOL

"""The tile kinds that the training calls choose for larger shapes: each case says
which kernels it has to reach (the names of what was launched are read back), so
that a changed choice cannot leave one untested.

Kernels are grouped_kernel<CTAs, columns, A across its rows, B across its rows,
epilogue, rows a CTA, sets>; epilogues: 0 rows, 1 weight gradient, 2 Newton-Schulz,
3 GELU and 4 SwiGLU hidden gradients, 5 rows over a long contraction.
"""
import re
import warnings

import pytest
import torch

import mixture_experts_layer_54_b200 as moe
from test_gpu_training import (BF, F32, F64, NS_TOL, QUINTIC, ffn_case, ffn_reference, newton_schulz,
                               randn, table, within)

pytestmark = pytest.mark.gpu

RAGGED = [257, 129, 0, 300, 255, 256, 1, 402]   # 200 rows a group


def launched(call):
    """(result, [template arguments of every grouped kernel that ran, in turn]; None
    where the machine lets nobody trace kernels)."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as prof:
        out = call()
        torch.cuda.synchronize()
    if not any("kernel" in e.name for e in prof.events()):
        warnings.warn("the profiler reports no kernels here: the tile kinds are not checked")
        return out, None
    runs = sorted((e.time_range.start, e.name) for e in prof.events() if "grouped_kernel<" in e.name)
    word = {"true": 1, "false": 0}
    args = [re.search(r"grouped_kernel<([^>]*)>", name).group(1) for _, name in runs]
    return out, [tuple(word[a] if a in word else int(a)
                       for a in re.sub(r"\(\w+\)| ", "", text).split(",")) for text in args]


@pytest.mark.parametrize("aligned,wide", [(False, 1288), (True, 1016)])
def test_products_on_pairs_of_sms(aligned, wide):
    """256 x 256 tiles of ragged groups, odd widths, NaN beside every group."""
    K = 328
    off, rows, R, spans = table(RAGGED, aligned)
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    for lo, hi in spans:
        inside[lo:hi] = True
    x, dy = randn(R, K, seed=1), randn(R, wide, seed=2)
    x[~inside] = float("nan")
    dy[~inside] = float("nan")
    W = randn(8, wide, K, seed=3, scale=K ** -0.5)
    Wx = randn(8, K, wide, seed=4, scale=K ** -0.5)
    y = torch.full((R, wide), 7.0, dtype=BF, device="cuda")
    dx = torch.full((R, wide), 7.0, dtype=BF, device="cuda")
    ws = moe.workspace(moe.lib().moe_grouped_workspace_size(1, 8, R, wide, K), "cuda")
    ws.fill_(255)
    _, kind = launched(lambda: moe.moe_grouped_matmul(x, W, off, rows, y=y, ws=ws))
    assert kind in (None, [(2, 256, 0, 0, 0, 128, 1)])
    assert moe.moe_device_status(ws) == 0
    _, kind = launched(lambda: moe.moe_grouped_matmul_dx(x, Wx, off, rows, dx=dx, ws=ws))
    assert kind in (None, [(2, 256, 0, 1, 0, 128, 1)])
    assert moe.moe_device_status(ws) == 0
    dW, kind = launched(lambda: moe.moe_grouped_matmul_dw(dy, x, off, rows, out_dtype=F32, ws=ws))
    assert kind in (None, [(2, 256, 1, 1, 1, 128, 1)])
    assert moe.moe_device_status(ws) == 0
    assert (y[~inside] == 7.0).all() and (dx[~inside] == 7.0).all()
    for g, (lo, hi) in enumerate(spans):
        a, b = x[lo:hi].to(F64), dy[lo:hi].to(F64)
        for got, w in ((y, W[g].to(F64).T), (dx, Wx[g].to(F64))):
            r = a @ w
            within(got[lo:hi], r, 2.0 ** -8 * r.abs() + K * 2.0 ** -23 * (a.abs() @ w.abs()))
        r = b.T @ a
        within(dW[g], r, 2.0 ** -24 * r.abs() + (hi - lo + 1) * 2.0 ** -23 * (b.abs().T @ a.abs()))


@pytest.mark.parametrize("N,K,epi", [(264, 3000, 0), (520, 320, 0), (136, 8200, 5), (1160, 8264, 5)])
def test_few_rows_on_tiles_of_32(N, K, epi):
    """Groups below, at and just past 32 rows, whole tiles and cut ones, in one
    accumulator and in several."""
    off, _, R, spans = table([20, 0, 9, 33, 2, 32, 1, 5, 16, 7], False)
    x, dy = randn(R, K, seed=1), randn(R, K, seed=2)
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    for lo, hi in spans:
        inside[lo:hi] = True
    x[~inside] = float("nan")
    dy[~inside] = float("nan")
    W = randn(10, N, K, seed=3, scale=K ** -0.5)
    Wx = randn(10, K, N, seed=4, scale=K ** -0.5)
    y, dx = (torch.full((R, N), 7.0, dtype=BF, device="cuda") for _ in range(2))
    _, kind = launched(lambda: moe.moe_grouped_matmul(x, W, off, y=y))
    assert kind in (None, [(1, 128, 0, 0, epi, 32, 1)])
    _, kind = launched(lambda: moe.moe_grouped_matmul_dx(dy, Wx, off, dx=dx))
    assert kind in (None, [(1, 128, 0, 1, epi, 32, 1)])
    assert (y[~inside] == 7.0).all() and (dx[~inside] == 7.0).all()
    for g, (lo, hi) in enumerate(spans):
        for got, a, w in ((y, x[lo:hi].to(F64), W[g].to(F64).T), (dx, dy[lo:hi].to(F64), Wx[g].to(F64))):
            r = a @ w
            within(got[lo:hi], r, 2.0 ** -8 * r.abs() + K * 2.0 ** -23 * (a.abs() @ w.abs()))


FFN = {
    # E, sizes, d, F, act, S, Fs, kernels of the call
    "swiglu_single": (40, [70, 1, 139, 70, 0] * 8, 128, 256, 1, 0, 0,
                      [(1, 128, 0, 0, 4, 128, 2), (1, 128, 0, 1, 0, 128, 1), (1, 128, 1, 1, 1, 128, 6)]),
    "gelu_single": (40, [70, 1, 139, 70, 0] * 8, 128, 256, 0, 1, 64,
                    [(1, 128, 0, 0, 3, 128, 2), (1, 128, 0, 1, 0, 128, 2), (1, 128, 1, 1, 1, 128, 6)]),
    "swiglu_pairs": (8, RAGGED, 1344, 256, 1, 1, 64,
                     [(2, 128, 0, 0, 4, 128, 2), (2, 256, 0, 1, 0, 128, 2), (2, 256, 1, 1, 1, 128, 6)]),
    "gelu_pairs": (8, RAGGED, 1344, 256, 0, 2, 64,
                   [(2, 128, 0, 0, 3, 128, 2), (2, 256, 0, 1, 0, 128, 2), (2, 256, 1, 1, 1, 128, 6)]),
    "swiglu_pairs_alone": (8, RAGGED, 1344, 320, 1, 0, 0,
                           [(2, 128, 0, 0, 4, 128, 2), (2, 256, 0, 1, 0, 128, 1),
                            (2, 256, 1, 1, 1, 128, 6)]),
    # du W1 + dv W3 past 8192 of contraction
    "swiglu_long_single": (4, [90, 70, 40, 33], 64, 4160, 1, 1, 64,
                           [(1, 128, 0, 0, 4, 128, 2), (1, 128, 0, 1, 5, 128, 2),
                            (1, 128, 1, 1, 1, 128, 6)]),
    "gelu_long_pairs": (8, RAGGED, 1344, 8256, 0, 2, 64,
                        [(2, 128, 0, 0, 3, 128, 2), (2, 256, 0, 1, 5, 128, 2),
                         (2, 256, 1, 1, 1, 128, 6)]),
    "swiglu_long_pairs_alone": (8, RAGGED, 1344, 4160, 1, 0, 0,
                                [(2, 128, 0, 0, 4, 128, 2), (2, 256, 0, 1, 5, 128, 1),
                                 (2, 256, 1, 1, 1, 128, 6)]),
    "gelu_long_single_alone": (4, [90, 70, 40, 33], 64, 8256, 0, 0, 0,
                               [(1, 128, 0, 0, 3, 128, 2), (1, 128, 0, 1, 5, 128, 1),
                                (1, 128, 1, 1, 1, 128, 6)]),
}


@pytest.mark.parametrize("name", list(FFN))
def test_ffn_gradients_of_every_tile_kind(name):
    E, sizes, d, F, act, S, Fs, want = FFN[name]
    cfg, x, off, kept, dY, W, sh, spans, inside = ffn_case(sum(sizes), d, E, 1, F, act, S, Fs, 1, sizes)
    dx = torch.full_like(x, 7.0)
    ws = moe.workspace(moe.moe_ffn_backward_workspace_size(cfg), "cuda")
    ws.fill_(255)
    g, kinds = launched(lambda: moe.moe_expert_ffn_backward(cfg, x, off, kept, dY, *W, **sh, dx_perm=dx,
                                                            dw_dtype=F32, ws=ws))
    assert kinds in (None, want)
    assert moe.moe_device_status(ws) == 0
    assert (dx[~inside] == 7.0).all()
    for e, (lo, hi) in enumerate(spans):
        ref, bound, _ = ffn_reference(x[lo:hi], dY[lo:hi], W[0][e], W[1][e] if act else None, W[2][e], act)
        got = (dx[lo:hi], g.dW1[e], g.dW3[e] if act else None, g.dW2[e])
        for what, a, r, b in zip(("dx", "dW1", "dW3", "dW2"), got, ref, bound):
            if r is not None:
                within(a, r, b, f"{what}[{e}]")
    dxs, bxs = 0, 0
    for s in range(S):
        ref, bound, bx = ffn_reference(sh["x"], sh["dY_shared"], sh["Ws1"][s],
                                       sh["Ws3"][s] if act else None, sh["Ws2"][s], act)
        dxs, bxs = dxs + ref[0], bxs + S * bx
        for what, a, r, b in zip(("dWs1", "dWs3", "dWs2"), (g.dWs1, g.dWs3, g.dWs2), ref[1:], bound[1:]):
            if r is not None:
                within(a[s], r, b, f"{what}[{s}]")
    if S:
        within(g.dx_shared, dxs, 2.0 ** -8 * dxs.abs() + (1 + 2.0 ** -8) * bxs, "dx_shared")


@pytest.mark.parametrize("E,m,n,kinds", [
    (60, 255, 400, {(2, 256, 0, 0, 2, 128, 1), (2, 256, 0, 1, 2, 128, 1)}),
    (60, 400, 255, {(2, 256, 1, 1, 2, 128, 1), (2, 256, 0, 0, 2, 128, 1)}),
    (74, 250, 131, {(2, 256, 1, 1, 2, 128, 1), (2, 256, 0, 0, 2, 128, 1)}),
    (70, 300, 520, {(1, 128, 0, 0, 2, 128, 1)})])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_stacks_of_every_tile_kind(E, m, n, kinds, dtype):
    """Mirrored halves, the low term and odd pitches on pairs of SMs."""
    G = randn(E, m, n, seed=m, dtype=dtype, scale=1e-3)
    ws = moe.workspace(moe.moe_orthogonalize_workspace_size(E, m, n, 5), "cuda")
    ws.fill_(255)
    U, ran = launched(lambda: moe.moe_orthogonalize(G, ws=ws))
    assert ran is None or (len(ran) == 15 and kinds <= set(ran)), ran
    assert moe.moe_device_status(ws) == 0
    ref = newton_schulz(G, 5, QUINTIC)
    rel = (U.to(F64) - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert rel.max().item() <= NS_TOL

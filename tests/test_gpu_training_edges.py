"""Edges of the training calls: what an earlier launch left in a workspace, sums
over very long contractions, updates far below eps, and the promised accuracy."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_54_b200 as moe
from mixture_experts_layer_54_b200 import _abi
from test_gpu_training import BF, F32, F64, NS_TOL, QUINTIC, ffn_case, newton_schulz, randn, table, within

pytestmark = pytest.mark.gpu


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


TAG_AT = 56   # of ParamsOf in csrc/grouped.cuh: the launch's tag in the counters


def launch_tags(graph):
    """Tags of the grouped kernels of a captured graph, from their arguments."""
    cu = ctypes.CDLL("libcuda.so.1")
    g, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(g, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(g, nodes, ctypes.byref(n)) == 0
    tags = []
    for node in nodes:
        kind = ctypes.c_int()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:   # a kernel
            continue
        p = KernelNode()
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        if p.block[0] in (320, 352):   # ten or eleven warps: the grouped kernel
            first = ctypes.c_void_p.from_address(p.params).value
            tags.append(ctypes.c_uint64.from_address(first + TAG_AT).value)
    return tags


def capture(call):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        out = call()
    tags = launch_tags(g)
    g.instantiate()
    return g, out, tags


@pytest.mark.parametrize("kind", ["y", "dx", "dw", "few"])
def test_counters_left_by_a_launch_that_gave_up(kind):
    """A replayed launch has the tag of the replay before.  Counters as one leaves
    them whose parts did not all arrive must not count as this launch's own."""
    sizes, N, K = {"y": ([600], 256, 4096), "dx": ([600], 4096, 256), "dw": ([9000], 128, 128),
                   "few": ([5, 40], 136, 8192)}[kind]
    off, _, R, spans = table(sizes, False)
    G = len(sizes)
    x, dy = randn(R, K, seed=1), randn(R, N, seed=2)
    W = randn(G, N, K, seed=3, scale=K ** -0.5)
    ws = moe.workspace(moe.lib().moe_grouped_workspace_size(1, G, R, N, K), "cuda")
    out = {"y": torch.zeros_like(dy), "few": torch.zeros_like(dy), "dx": torch.zeros_like(x),
           "dw": torch.zeros((G, N, K), dtype=F32, device="cuda")}[kind]
    call = {"y": lambda: moe.moe_grouped_matmul(x, W, off, y=out, ws=ws),
            "dx": lambda: moe.moe_grouped_matmul_dx(dy, W, off, dx=out, ws=ws),
            "dw": lambda: moe.moe_grouped_matmul_dw(dy, x, off, dW=out, ws=ws)}
    call = call["y" if kind == "few" else kind]
    graph, _, tags = capture(call)
    assert len(tags) == 1 and tags[0] != 0
    counters = ws[256:256 + (16 << 10)].view(torch.int64)
    for seed, arrived in enumerate((1, 2, 3, 4, 6, 9, 15), 4):
        x.copy_(randn(R, K, seed=seed))
        dy.copy_(randn(R, N, seed=seed + 20))
        out.zero_()
        call()
        want = out.clone()
        out.zero_()
        left = tags[0] << 16 | arrived
        counters.fill_(left - (1 << 64) if left >> 63 else left)
        graph.replay()
        torch.cuda.synchronize()
        assert moe.moe_device_status(ws) == 0
        assert torch.equal(out, want)


def test_a_tail_behind_seconds_of_work():
    """About three seconds of whole tiles, then one group that ends inside a step of
    16 rows: the wait for its tail is not longer than a stage.  (The even groups all
    have the same rows, or so much work would not fit in memory.)"""
    R, N, K, G = 7 << 17, 8192, 2048, 255
    x = torch.empty((R, K), dtype=BF, device="cuda").bernoulli_(0.5)
    dy = torch.empty((R, N), dtype=BF, device="cuda").bernoulli_(0.5)
    off = torch.zeros(G + 1, dtype=torch.int32)
    off[1::2] = R
    rows = torch.full((G,), R, dtype=torch.int32)
    rows[-1] = 7
    ws = moe.workspace(moe.lib().moe_grouped_workspace_size(1, G, R, N, K), "cuda")
    dW = moe.moe_grouped_matmul_dw(dy, x, off.cuda(), rows.cuda(), ws=ws)
    assert moe.moe_device_status(ws) == 0
    assert torch.equal(dW[-1].float(), dy[:7].float().T @ x[:7].float())   # whole numbers up to 7
    for g in range(1, G - 1):
        assert torch.equal(dW[g], dW[0]) if g % 2 == 0 else not dW[g].any()


def half_step(ref):
    """Half a bf16 step at every element."""
    return torch.ldexp(torch.ones_like(ref), torch.frexp(ref)[1] - 9)


@pytest.mark.parametrize("R,N,K,G", [(60, 264, 1 << 17, 1), (5, 136, 1 << 20, 1), (200, 128, 1 << 18, 2),
                                     (600, 4000, 1 << 15, 1), (1600, 1288, 14336, 8)])
def test_products_over_long_contractions(R, N, K, G):
    """Sums of values of one sign, where every truncation counts: 8192 of them in one
    accumulator (512 steps of 16, each truncated), up to 128 of those added up and
    16 parts of a tile, all relative to the sum."""
    off, _, rows, spans = table([R // G] * G, False)
    x = randn(rows, K, seed=1).abs()
    W = randn(G, N, K, seed=3, scale=K ** -0.5).abs()
    Wt = W.mT.contiguous()
    y = moe.moe_grouped_matmul(x, W, off)
    dx = moe.moe_grouped_matmul_dx(x, Wt, off)   # [G, K, N]: the same sums, W read across its rows
    tol = (512 + math.ceil(K / 8192) + 16) * 2.0 ** -23
    for g, (lo, hi) in enumerate(spans):
        ref = x[lo:hi].to(F64) @ W[g].to(F64).T
        for got in (y, dx):
            within(got[lo:hi], ref, half_step(ref) + tol * ref)


# the promised error of five steps, and one rounding to bf16
PROMISED = 2e-3 + 2.0 ** -8
CUBIC = (1.5, -0.5, 0.0)


@pytest.mark.parametrize("m,n", [(48, 80), (90, 40), (300, 700), (520, 264), (8, 700), (900, 33)])
@pytest.mark.parametrize("steps,coeffs,tol", [(1, QUINTIC, PROMISED), (2, QUINTIC, PROMISED),
                                              (5, QUINTIC, PROMISED), (30, CUBIC, NS_TOL)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_orthogonalize_far_below_eps(m, n, steps, coeffs, tol, dtype):
    """|G| from eps down to 1e-24 eps: the result is a to the number of steps times
    |G| / eps, small but not nothing, until the steps have brought it near 1."""
    eps = 1e-7
    G = torch.stack([randn(m, n, seed=i, dtype=F32) for i in range(7)])
    sizes = torch.tensor([1.0, 1e-3, 1e-6, 1e-9, 1e-12, 1e-18, 1e-24], device="cuda")
    G = (G / G.flatten(1).norm(dim=1)[:, None, None] * (eps * sizes)[:, None, None]).to(dtype)
    U = moe.moe_orthogonalize(G, steps=steps, coeffs=coeffs, eps=eps)
    ref = newton_schulz(G, steps, coeffs, eps)
    for e in range(len(sizes)):
        rel = ((U[e].to(F64) - ref[e]).norm() / ref[e].norm()).item()
        assert rel <= tol, (e, rel)


@pytest.mark.parametrize("coeffs,steps,last", [((2.79, 0.0, 0.0), 2, 2.79 ** 2), ((1.0, 29.5, 0.0), 1, 30.5),
                                               ((0.0, 0.0, 1.3), 2, 1.3 ** 6), ((-30.9, 0.0, 0.0), 1, -30.9)])
@pytest.mark.parametrize("m,n", [(40, 64), (300, 264), (20, 600)])
def test_orthogonalize_at_the_edge_of_its_range(coeffs, steps, last, m, n):
    """Coefficients just inside what is refused, on a matrix of one singular value,
    which the norm makes 1: nothing overflows.  (X, B and the product: each operand
    is off by at most 2^-11, five times over for the fifth power.)"""
    u, v = randn(2, m, 1, seed=1, dtype=F32), randn(2, 1, n, seed=2, dtype=F32)
    G = u @ v
    U = moe.moe_orthogonalize(G, steps=steps, coeffs=coeffs, eps=0.0)
    ref = last * G.to(F64) / torch.linalg.matrix_norm(G.to(F64))[:, None, None]
    for e in range(2):
        assert ((U[e].to(F64) - ref[e]).norm() / ref[e].norm()).item() <= 2.0 ** -8 + 20 * 2.0 ** -11


def update(kind, E, m, n, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(m * n)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    if kind == "noise":
        G = r(E, m, n)
    elif kind == "rank_32":
        G = r(E, m, 32) @ r(E, 32, n)
    else:   # singular values 1, 1/2, 1/3, ...
        p = min(m, n)
        u, v = torch.linalg.qr(r(E, m, p))[0], torch.linalg.qr(r(E, n, p))[0]
        G = (u / torch.arange(1, p + 1, device="cuda")) @ v.mT
    return (1e-3 * G).to(dtype)


@pytest.mark.parametrize("kind", ["noise", "rank_32", "decaying"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n", [(300, 700), (520, 264), (1024, 512), (130, 2100), (2000, 160)])
def test_orthogonalize_keeps_its_promise(m, n, dtype, kind):
    """2e-3 in 2-norm, and the rounding to bf16: at most half a step, evenly spread,
    so 2^-8 / sqrt(3) of the norm."""
    G = update(kind, 2, m, n, dtype)
    U, ref = moe.moe_orthogonalize(G), newton_schulz(G, 5, QUINTIC)
    for e in range(2):
        rel = ((U[e].to(F64) - ref[e]).norm() / ref[e].norm()).item()
        assert rel <= 2e-3 + 2.0 ** -8 / math.sqrt(3), (e, rel)


@pytest.mark.parametrize("kind", ["noise", "rank_32", "decaying"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n", [(128, 320), (48, 80), (320, 128), (34, 33)])
def test_orthogonalize_of_small_matrices_is_as_in_fp32(m, n, dtype, kind):
    """Terms of 22 bits: 2e-2 for 11 bits in the worst kind, so 1e-5 for 22.  What an
    element is off by beyond half a bf16 step is at most twice its error before the
    rounding (twice, where the step doubles)."""
    G = update(kind, 2, m, n, dtype)
    U, ref = moe.moe_orthogonalize(G).to(F64), newton_schulz(G, 5, QUINTIC)
    half = half_step(ref)
    for e in range(2):
        over = ((U[e] - ref[e]).abs() - half[e]).clamp(min=0).norm() / ref[e].norm()
        assert over.item() <= 2e-5, (e, over.item())


def test_a_wait_that_ran_out_is_not_lost_with_its_workspace():
    """A bounded wait of the training kernels, given 50 ms on a barrier that nothing
    arrives on: the status stays through later calls that make their own workspace,
    until it is cleared, and the calls go on."""
    assert moe.moe_training_status() == 0
    moe.moe_probe_training_timeout(50_000_000)
    off, _, R, spans = table([60, 40], False)
    x, W = randn(R, 64, seed=1), randn(2, 72, 64, seed=2, scale=1 / 8)
    G = randn(2, 48, 40, seed=3)
    y, U = moe.moe_grouped_matmul(x, W, off), moe.moe_orthogonalize(G)
    assert moe.moe_training_status() == _abi.MOE_ERR_DEVICE_TIMEOUT
    moe.moe_clear_training_status()
    assert torch.equal(moe.moe_grouped_matmul(x, W, off)[3:103], y[3:103])
    assert torch.equal(moe.moe_orthogonalize(G), U)
    assert moe.moe_training_status() == 0


LONG_AND_NARROW = [(4, 637), (637, 4), (1, 5000), (5000, 1), (17, 330), (56, 4096), (1001, 55), (330, 33),
                   (2, 100001), (9, 321), (16, 2049), (513, 32)]


@pytest.mark.parametrize("kind", ["noise", "rank_32", "decaying", "equal"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n", LONG_AND_NARROW)
def test_orthogonalize_of_few_rows_or_columns(m, n, dtype, kind):
    """Up to 56 rows or columns, longer than one block holds: singular values that lie
    together (all of them, or equal) are no worse than others.  The last product is in
    fp32: P, up to 485 after five steps, times X, at 2^-24 each and a few of them."""
    E = 5
    if kind == "equal":
        g = torch.Generator(device="cuda")
        g.manual_seed(m + n)
        G = torch.linalg.qr(torch.randn((E, max(m, n), min(m, n)), generator=g, device="cuda"))[0]
        G = (G if m > n else G.mT).to(dtype).contiguous()
    else:
        G = update(kind, E, m, n, dtype)
    ws = moe.workspace(moe.moe_orthogonalize_workspace_size(E, m, n), "cuda")
    ws.fill_(255)
    U, ref = moe.moe_orthogonalize(G, ws=ws).to(F64), newton_schulz(G, 5, QUINTIC)
    assert moe.moe_device_status(ws) == 0
    half = half_step(ref)
    for e in range(E):
        over = ((U[e] - ref[e]).abs() - half[e]).clamp(min=0).norm() / ref[e].norm()
        assert over.item() <= 2e-4, (e, over.item())


@pytest.mark.parametrize("m,n", [(8, 700), (700, 8), (50, 400), (40, 60), (300, 520)])
@pytest.mark.parametrize("steps,coeffs", [(6, QUINTIC), (7, QUINTIC), (32, QUINTIC), (32, CUBIC)])
def test_orthogonalize_of_low_rank_by_many_steps(m, n, steps, coeffs):
    """Directions that G does not have are multiplied by a in every step, whatever the
    rounding left there: with more steps than precision they come out as singular
    values near 1, never larger.  (The quintic's stay below 1.21, the cubic's below 1;
    a singular value past 1.25 is an overflow on its way.)"""
    G = randn(3, m, 2, seed=1, dtype=F32) @ randn(3, 2, n, seed=2, dtype=F32)
    U = moe.moe_orthogonalize(G, steps=steps, coeffs=coeffs)
    assert torch.isfinite(U).all()
    assert torch.linalg.svdvals(U.to(F64)).max().item() <= 1.25


@pytest.mark.parametrize("m,n", [(7, 700), (700, 7), (50, 400), (57, 400)])
def test_few_rows_or_columns_of_zeros_infinities_and_far_magnitudes(m, n):
    G = randn(6, m, n, seed=1, dtype=F32)
    G[1] = 0
    G[2, 3, 4] = float("inf")
    G[3] *= 2.0 ** -130
    G[4] *= 2.0 ** 110
    U = moe.moe_orthogonalize(G, eps=0.0)
    assert torch.isnan(U[1]).all() and torch.isnan(U[2]).all()
    ref = newton_schulz(G, 5, QUINTIC, eps=0.0)
    close, far = 2.0 ** -8 + 1e-4, NS_TOL
    tol = close if min(m, n) <= 56 else far
    for e in (0, 3, 4, 5):
        assert ((U[e].to(F64) - ref[e]).norm() / ref[e].norm()).item() <= tol
    assert (moe.moe_orthogonalize(G[1:2]) == 0).all()
    # one matrix, in and out off the 16-byte grid; scale; one step and many; a replay
    size = m * n
    flat, out = (torch.zeros(size + 1, dtype=BF, device="cuda") for _ in range(2))
    flat[1:] = G[0].reshape(-1).to(BF)
    one = flat[1:].view(m, n)
    for steps, coeffs, scale in ((1, QUINTIC, 1.0), (5, QUINTIC, 0.3), (30, CUBIC, 1.0)):
        got = moe.moe_orthogonalize(one, steps=steps, coeffs=coeffs, scale=scale, U=out[1:].view(m, n))
        ref = scale * newton_schulz(one, steps, coeffs)
        many = coeffs[0] ** steps > 2048
        assert ((got.to(F64) - ref).norm() / ref.norm()).item() <= (far if many else tol)
        graph, again, _ = capture(lambda: moe.moe_orthogonalize(one, steps=steps, coeffs=coeffs, scale=scale))
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, got)

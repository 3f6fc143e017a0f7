"""Cases of the expert training operators: what is measured, the operators in plain torch, and
their definition in 64 bits.

  product        y[r] = W[g] x[r] for the rows r of each group g (one weight matrix per expert)
  product_dx     dx[r] = W[g]^T dy[r]
  product_dw     dW[g] = sum over the rows r of group g of dy[r] x[r]^T, alone or added to dW
  combine_grad   gradients of the gated combine: dY_perm[row] = gate * dy[token] and
                 dgates[t, j] = <dy[t], Y_perm[row]>
  ffn_grad       gradients of the expert FFNs (GELU or SwiGLU, shared experts too), with the hidden
                 activations computed again from x
  orthogonalize  five Newton-Schulz steps on every expert's update

A group's rows are consecutive.  "packed": group g + 1 begins where group g ends.  "aligned":
groups begin on multiples of 128 rows, as the layer's capacity step lays them out, and the rows
between a group's end and the next group's start belong to nobody.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NS_COEFFS = (3.4445, -4.7750, 2.0315)   # quintic of the Newton-Schulz step
NS_STEPS = 5
NS_EPS = 1e-7


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decode step of 8 tokens, top-2 of 8 experts, through the second matrix of the
        # Mixtral-shaped experts: two rows an expert on average, the weights are the work.
        dict(name="product_decode", op="product", dtype="bf16", G=8, rows=16, N=4096, K=14336,
             cap=8, skew=0.0, layout=1, aligned=False),
        # A training batch through the first matrix of the DeepSeekMoE-shaped experts: many small
        # experts, ragged, on the layer's 128-row boundaries.
        dict(name="product_batch", op="product", dtype="bf16", G=64, rows=98304, N=512, K=1024,
             cap=2304, skew=0.3, layout=2, aligned=True),
        # Input gradient in the fp32 layer of the tests: latency alone.
        dict(name="dx_tiny", op="product_dx", dtype="fp32", G=4, rows=128, N=64, K=32,
             cap=40, skew=0.2, layout=3, aligned=False),
        # Input gradient through the first matrix of the Mixtral-shaped experts: the largest product.
        dict(name="dx_batch", op="product_dx", dtype="bf16", G=8, rows=16384, N=14336, K=4096,
             cap=2560, skew=0.2, layout=4, aligned=True),
        # Weight gradient of the Switch-shaped experts, packed groups of odd lengths.
        dict(name="dw_packed", op="product_dw", dtype="bf16", G=8, rows=4096, N=4096, K=1024,
             cap=768, skew=0.2, layout=5, aligned=False, out="bf16", add=False),
        # Weight gradient of the DeepSeekMoE-shaped experts added in fp32 to what earlier
        # micro-batches left.
        dict(name="dw_add", op="product_dw", dtype="bf16", G=64, rows=98304, N=512, K=1024,
             cap=2304, skew=0.3, layout=6, aligned=True, out="fp32", add=True),
        # The combine's gradient for a few tokens of the fp32 layer, and for the DeepSeekMoE-shaped
        # batch, some of whose assignments the capacity limit dropped.
        dict(name="combine_tiny", op="combine_grad", dtype="fp32", T=64, d=32, E=4, k=2, cap=40),
        dict(name="combine_batch", op="combine_grad", dtype="bf16", T=16384, d=1024, E=64, k=6,
             cap=1700),
        # The gradients of the Switch-shaped layer's GELU experts.
        dict(name="ffn_gelu", op="ffn_grad", dtype="bf16", T=4096, d=1024, E=8, k=1, d_ff=4096,
             act=0, n_shared=0, d_ff_shared=0, cap=512, skew=0.2, layout=7),
        # The gradients of the DeepSeekMoE-shaped layer's SwiGLU experts with two shared experts.
        dict(name="ffn_swiglu", op="ffn_grad", dtype="bf16", T=16384, d=1024, E=64, k=6, d_ff=512,
             act=1, n_shared=2, d_ff_shared=512, cap=2304, skew=0.3, layout=8),
        # The update of the fp32 layer's experts, and of the Switch-shaped experts' first matrices.
        dict(name="orthogonalize_tiny", op="orthogonalize", dtype="fp32", E=4, m=64, n=32),
        dict(name="orthogonalize_stack", op="orthogonalize", dtype="bf16", E=8, m=4096, n=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = 2e12   # flops of a drawn case; the largest listed one has 1.9e12
    op = rng.choice(["product", "product_dx", "product_dw", "combine_grad", "ffn_grad",
                     "orthogonalize"])
    layout = rng.randrange(1 << 20)
    if op.startswith("product"):
        if rng.random() < 0.2:   # the fp32 layer: small, any size
            case = dict(op=op, dtype="fp32", G=rng.randint(1, 8), rows=_log_int(rng, 1, 500),
                        N=_log_int(rng, 5, 200), K=_log_int(rng, 5, 200))
        else:
            while True:
                case = dict(op=op, dtype="bf16", G=_log_int(rng, 1, 64),
                            rows=_log_int(rng, 1, 60000), N=8 * _log_int(rng, 8, 900),
                            K=8 * _log_int(rng, 8, 900))
                weights = case["G"] * case["N"] * case["K"]
                if 2 * case["rows"] * case["N"] * case["K"] < most / 4 and weights < 4e8:
                    break
        mean = case["rows"] / case["G"]
        case.update(cap=max(1, int(mean * rng.uniform(1.2, 2.0) + 2)), skew=rng.uniform(0, 0.5),
                    layout=layout, aligned=rng.random() < 0.5)
        if op == "product_dw":
            out = "fp32" if case["dtype"] == "fp32" else rng.choice(["bf16", "fp32"])
            case.update(out=out, add=rng.random() < 0.5)
        return case
    if op == "combine_grad":
        E = _log_int(rng, 2, 128)
        k = rng.randint(1, min(E, 8))
        T = _log_int(rng, 1, 16384)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), T=T,
                    d=64 * _log_int(rng, 1, 16), E=E, k=k,
                    cap=max(1, int(rng.uniform(1.0, 2.0) * T * k / E + 1)))
    if op == "ffn_grad":
        while True:
            E = _log_int(rng, 1, 64)
            case = dict(op=op, dtype="bf16", T=_log_int(rng, 1, 16384), d=64 * _log_int(rng, 1, 32),
                        E=E, k=rng.randint(1, min(E, 6)), d_ff=64 * _log_int(rng, 1, 64),
                        act=rng.randint(0, 1), n_shared=rng.choice([0, 0, 1, 2]), d_ff_shared=0)
            case["d_ff_shared"] = 64 * _log_int(rng, 1, 16) if case["n_shared"] else 0
            case.update(cap=max(1, int(1.5 * case["T"] * case["k"] / E + 2)),
                        skew=rng.uniform(0, 0.5), layout=layout)
            if work(case)["flops"] < most / 3 and E * case["d"] * case["d_ff"] < 1.5e8:
                return case
    while True:
        case = dict(op=op, dtype=rng.choice(["bf16", "fp32"]), E=_log_int(rng, 1, 64),
                    m=_log_int(rng, 16, 4096), n=_log_int(rng, 16, 4096))
        if work(case)["flops"] < most / 4:
            return case


# ------------------------------------------------------------------ layouts

def _sizes(G, rows, cap, skew, layout):
    """Rows of each group: `rows` draws over G groups of unequal weight, each held at `cap`."""
    rng = np.random.RandomState(layout % (1 << 31))
    p = (1.0 + np.arange(G)) ** -skew
    p = rng.permutation(p / p.sum())
    return np.minimum(rng.multinomial(rows, p), cap)


def _offsets(sizes, aligned):
    """G + 1 starts and the number of rows of the buffers."""
    spans = -(-sizes // 128) * 128 if aligned else sizes
    off = np.concatenate([[0], np.cumsum(spans)])
    return off, int(off[-1])


def _groups(case):
    sizes = _sizes(case["G"], case["rows"], case["cap"], case["skew"], case["layout"])
    off, R = _offsets(sizes, case["aligned"])
    return sizes, off, R


def _ffn_groups(case):
    sizes = _sizes(case["E"], case["T"] * case["k"], min(case["cap"], case["T"]), case["skew"],
                   case["layout"])
    off, R = _offsets(sizes, True)
    return sizes, off, R


def _dev(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _perm_rows(case):
    kept = min(case["T"] * case["k"], min(case["cap"], case["T"]) * case["E"])
    return -(-(kept + case["E"] * 127) // 128) * 128


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype="bf16", scale=1.0):
        t = torch.randn(shape, generator=g, device="cuda")
        return (t * scale).to(DTYPES[dtype])

    op, dt = case["op"], case["dtype"]
    s = {"case": case}
    if op.startswith("product"):
        sizes, off, R = _groups(case)
        G, N, K = case["G"], case["N"], case["K"]
        s.update(R=R, cap=int(sizes.max()), offsets=_dev(off), rows=_dev(sizes))
        if op != "product_dw":
            s["W"] = randn(G, N, K, dtype=dt, scale=1 / math.sqrt(K))
        if op != "product_dx":
            s["x"] = randn(R, K, dtype=dt)
        if op != "product":
            s["dy"] = randn(R, N, dtype=dt, scale=1e-2)
        if op == "product":
            s["y"] = torch.zeros((R, N), dtype=DTYPES[dt], device="cuda")
        if op == "product_dx":
            s["dx"] = torch.zeros((R, K), dtype=DTYPES[dt], device="cuda")
        if op == "product_dw" and case["add"]:
            s["dW"] = randn(G, N, K, dtype=case["out"], scale=1e-1)
    elif op == "combine_grad":
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        bias = 0.5 * torch.randn((E,), generator=g, device="cuda")
        score = torch.randn((T, E), generator=g, device="cuda") + bias
        topk = score.topk(k, dim=1).indices
        hot = torch.nn.functional.one_hot(topk.reshape(-1), E)
        pos = ((hot.cumsum(0) - 1) * hot).sum(1).reshape(T, k)
        keep = pos < case["cap"]
        counts = hot.sum(0).clamp(max=case["cap"])
        off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
        off[1:] = ((counts + 127) // 128 * 128).cumsum(0)
        R = _perm_rows(case)
        s.update(R=R, topk=topk.int(), pos=pos.int(), keep=keep.to(torch.uint8), offsets=off.int(),
                 gates=torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1),
                 dy=randn(T, d, dtype=dt, scale=1e-2), Y_perm=randn(R, d, dtype=dt),
                 dY_perm=torch.zeros((R, d), dtype=DTYPES[dt], device="cuda"))
    elif op == "ffn_grad":
        sizes, off, used = _ffn_groups(case)
        T, d, E, F = case["T"], case["d"], case["E"], case["d_ff"]
        S, Fs, R = case["n_shared"], case["d_ff_shared"], _perm_rows(case)
        s.update(R=R, cap=int(sizes.max()), offsets=_dev(off), rows=_dev(sizes),
                 x_perm=randn(R, d), dY_perm=randn(R, d, scale=1e-2),
                 W1=randn(E, F, d, scale=1 / math.sqrt(d)), W2=randn(E, d, F, scale=1 / math.sqrt(F)),
                 W3=randn(E, F, d, scale=1 / math.sqrt(d)) if case["act"] else None,
                 dx_perm=torch.zeros((R, d), dtype=torch.bfloat16, device="cuda"))
        for name in ("x", "dy", "Ws1", "Ws2", "Ws3"):
            s[name] = None
        if S:
            s.update(x=randn(T, d), dy=randn(T, d, scale=1e-2),
                     Ws1=randn(S, Fs, d, scale=1 / math.sqrt(d)),
                     Ws2=randn(S, d, Fs, scale=1 / math.sqrt(Fs)),
                     Ws3=randn(S, Fs, d, scale=1 / math.sqrt(d)) if case["act"] else None)
    else:
        # an update as training gives it: a few strong directions over noise
        E, m, n = case["E"], case["m"], case["n"]
        r = min(8, m, n)
        u = torch.randn((E, m, r), generator=g, device="cuda")
        v = torch.randn((E, r, n), generator=g, device="cuda")
        noise = torch.randn((E, m, n), generator=g, device="cuda")
        s["G"] = (1e-3 * (0.5 * (u @ v) / math.sqrt(r) + noise)).to(DTYPES[dt])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"product": _plain_product, "product_dx": _plain_dx, "product_dw": _plain_dw,
            "combine_grad": _plain_combine, "ffn_grad": _plain_ffn,
            "orthogonalize": _plain_orthogonalize}[case["op"]](s, case)


def _run_own(s, case):
    import mixture_experts_layer_54_b200 as moe
    op = case["op"]
    if op == "product":
        return moe.moe_grouped_matmul(s["x"], s["W"], s["offsets"], s["rows"], y=s["y"])
    if op == "product_dx":
        return moe.moe_grouped_matmul_dx(s["dy"], s["W"], s["offsets"], s["rows"], dx=s["dx"])
    if op == "product_dw":
        return moe.moe_grouped_matmul_dw(s["dy"], s["x"], s["offsets"], s["rows"],
                                         add=s.get("dW"), out_dtype=DTYPES[case["out"]])
    if op == "combine_grad":
        cfg = moe.moe_config(T=case["T"], d=case["d"], E=case["E"], k=case["k"], d_ff=64, act=1,
                             dtype=int(case["dtype"] == "bf16"), cf=_cf(case))
        dY_perm, dgates = moe.moe_combine_backward(cfg, s["dy"], s["Y_perm"], s["gates"], s["topk"],
                                                   s["pos"], s["keep"], s["offsets"],
                                                   dY_perm=s["dY_perm"])
        return {"dY_perm": dY_perm, "dgates": dgates}
    if op == "ffn_grad":
        cfg = moe.moe_config(T=case["T"], d=case["d"], E=case["E"], k=case["k"], d_ff=case["d_ff"],
                             n_shared=case["n_shared"], d_ff_shared=case["d_ff_shared"],
                             act=case["act"], dtype=1, cf=_cf(case))
        r = moe.moe_expert_ffn_backward(cfg, s["x_perm"], s["offsets"], s["rows"], s["dY_perm"],
                                        s["W1"], s["W3"], s["W2"], x=s["x"], dY_shared=s["dy"],
                                        Ws1=s["Ws1"], Ws3=s["Ws3"], Ws2=s["Ws2"],
                                        dx_perm=s["dx_perm"])
        return _named(r.dx_perm, r.dW1, r.dW3, r.dW2, r.dx_shared, r.dWs1, r.dWs3, r.dWs2)
    return moe.moe_orthogonalize(s["G"], steps=NS_STEPS, coeffs=NS_COEFFS, eps=NS_EPS)


def _cf(case):
    """The capacity factor whose limit C is the case's (infinite where that holds every token)."""
    T, k, E, cap = case["T"], case["k"], case["E"], case["cap"]
    cf = (cap - 0.5) * E / (T * k)
    return cf if cap < T and cf >= 1.0 else (math.inf if cap >= T else 1.0)


def _named(dx, dW1, dW3, dW2, dxs=None, dWs1=None, dWs3=None, dWs2=None):
    out = dict(dx=dx, dW1=dW1, dW3=dW3, dW2=dW2, dx_shared=dxs, dWs1=dWs1, dWs3=dWs3, dWs2=dWs2)
    return {k: v for k, v in out.items() if v is not None}


# ------------------------------------------------------------------ plain forms

def _index(s):
    """Row of each (group, place), whether that place is taken, and the reverse for every row."""
    off, rows, R = s["offsets"].long(), s["rows"].long(), s["R"]
    place = torch.arange(s["cap"], device="cuda")
    taken = place[None, :] < rows[:, None]
    index = torch.where(taken, off[:-1, None] + place[None, :], 0)
    r = torch.arange(R, device="cuda")
    group = (torch.searchsorted(off, r, right=True) - 1).clamp(0, rows.numel() - 1)
    inside = r - off[group]
    mine = inside < rows[group]
    return index, taken, group, torch.where(mine, inside, 0), mine


def _pad(t, index, taken):
    return t.float()[index] * taken[:, :, None]


def _unpad(p, group, inside, mine, like):
    return torch.where(mine[:, None], p[group, inside].to(like.dtype), like)


def _plain_product(s, case):
    if s["R"] == 0:
        return s["y"]
    index, taken, group, inside, mine = _index(s)
    p = torch.bmm(_pad(s["x"], index, taken), s["W"].float().transpose(1, 2))
    return _unpad(p, group, inside, mine, s["y"])


def _plain_dx(s, case):
    if s["R"] == 0:
        return s["dx"]
    index, taken, group, inside, mine = _index(s)
    p = torch.bmm(_pad(s["dy"], index, taken), s["W"].float())
    return _unpad(p, group, inside, mine, s["dx"])


def _plain_dw(s, case):
    index, taken = _index(s)[:2]
    p = torch.bmm(_pad(s["dy"], index, taken).transpose(1, 2), _pad(s["x"], index, taken))
    if case["add"]:
        p = p + s["dW"].float()
    return p.to(DTYPES[case["out"]])


def _plain_combine(s, case):
    d = case["d"]
    keep = s["keep"].bool()
    # a dropped assignment has no row: it points at one past the last
    row = torch.where(keep, s["offsets"].long()[s["topk"].long()] + s["pos"].long(), s["R"])
    dy = s["dy"].float()
    wide = torch.cat([s["Y_perm"].float(), torch.zeros((1, d), device="cuda")])
    dgates = (wide[row] * dy[:, None, :]).sum(-1) * keep
    out = torch.cat([s["dY_perm"], s["dY_perm"][:1]])
    out[row.reshape(-1)] = (s["gates"][:, :, None] * dy[:, None, :]).reshape(-1, d).to(out.dtype)
    return {"dY_perm": out[:-1], "dgates": dgates}


def _act_grads(u, v, dh, act):
    """(h, du, dv) of h = gelu(u), or of h = silu(u) v."""
    if act == 0:
        cdf = 0.5 * (1 + torch.erf(u / math.sqrt(2)))
        return u * cdf, dh * (cdf + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)), None
    g = torch.sigmoid(u)
    return u * g * v, dh * v * g * (1 + u * (1 - g)), dh * u * g


def _plain_ffn_grads(x, dy, W1, W3, W2, act):
    """Gradients of y = W2 act(W1 x, W3 x) for x, dy [groups, rows, d] in 32 bits."""
    W1, W2 = W1.float(), W2.float()
    u = torch.bmm(x, W1.transpose(1, 2))
    v = torch.bmm(x, W3.float().transpose(1, 2)) if act else None
    h, du, dv = _act_grads(u, v, torch.bmm(dy, W2), act)
    dx = torch.bmm(du, W1)
    if act:
        dx = dx + torch.bmm(dv, W3.float())
    dW3 = torch.bmm(dv.transpose(1, 2), x) if act else None
    return dx, torch.bmm(du.transpose(1, 2), x), dW3, torch.bmm(dy.transpose(1, 2), h)


def _plain_ffn(s, case):
    act, bf16 = case["act"], torch.bfloat16
    index, taken, group, inside, mine = _index(s)
    dx, dW1, dW3, dW2 = _plain_ffn_grads(_pad(s["x_perm"], index, taken),
                                         _pad(s["dY_perm"], index, taken), s["W1"], s["W3"],
                                         s["W2"], act)
    out = [_unpad(dx, group, inside, mine, s["dx_perm"]), dW1, dW3, dW2]
    if case["n_shared"]:
        S = case["n_shared"]
        x = s["x"].float().expand(S, -1, -1)
        dy = s["dy"].float().expand(S, -1, -1)
        dxs, dWs1, dWs3, dWs2 = _plain_ffn_grads(x, dy, s["Ws1"], s["Ws3"], s["Ws2"], act)
        out += [dxs.sum(0), dWs1, dWs3, dWs2]
    return _named(*[None if t is None else t.to(bf16) for t in out])


def _plain_orthogonalize(s, case):
    a, b, c = NS_COEFFS
    X = s["G"].float()
    wide = case["m"] <= case["n"]
    X = X if wide else X.transpose(1, 2)
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        A = torch.bmm(X, X.transpose(1, 2))
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    return (X if wide else X.transpose(1, 2)).to(torch.bfloat16).contiguous()


# ------------------------------------------------------------------ the least work

def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("product"):
        sizes = _groups(case)[0]
        n, busy = int(sizes.sum()), int((sizes > 0).sum())
        N, K = case["N"], case["K"]
        flops = 2.0 * n * N * K
        if op == "product_dw":
            o = 2 if case["out"] == "bf16" else 4
            return {"bytes": e * n * (N + K) + o * case["G"] * N * K * (2 if case["add"] else 1),
                    "flops": flops}
        return {"bytes": e * (n * (N + K) + busy * N * K), "flops": flops}
    if op == "combine_grad":
        n = min(case["T"] * case["k"], case["cap"] * case["E"])
        d, T, k = case["d"], case["T"], case["k"]
        return {"bytes": e * (T * d + 2 * n * d) + T * k * 17, "flops": 3.0 * n * d}
    if op == "ffn_grad":
        sizes = _ffn_groups(case)[0]
        n, busy = int(sizes.sum()), int((sizes > 0).sum())
        d, F, E, T = case["d"], case["d_ff"], case["E"], case["T"]
        S, Fs = case["n_shared"], case["d_ff_shared"]
        mats = 3 if case["act"] else 2
        # per matrix: input gradient and weight gradient; the hidden activations once more
        products = 3 * mats - 1
        return {"bytes": 2 * (3 * n * d + mats * (busy + E) * d * F
                              + (3 * T * d + 2 * mats * S * d * Fs if S else 0)),
                "flops": 2.0 * products * d * (n * F + S * T * Fs)}
    m, n = sorted((case["m"], case["n"]))
    # X X^T and A A are symmetric: half of each
    return {"bytes": case["E"] * m * n * (e + 2),
            "flops": float(NS_STEPS * case["E"]) * (1.0 * m * m * n + 1.0 * m ** 3 + 2.0 * m * m * n)}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    if op.startswith("product"):
        sizes, off, R = _groups(case)
        spans = [(int(off[i]), int(off[i] + sizes[i])) for i in range(case["G"])]
        if op == "product":
            out = s["y"].to(f)
            for i, (lo, hi) in enumerate(spans):
                out[lo:hi] = s["x"][lo:hi].to(f) @ s["W"][i].to(f).T
        elif op == "product_dx":
            out = s["dx"].to(f)
            for i, (lo, hi) in enumerate(spans):
                out[lo:hi] = s["dy"][lo:hi].to(f) @ s["W"][i].to(f)
        else:
            out = torch.stack([s["dy"][lo:hi].to(f).T @ s["x"][lo:hi].to(f) for lo, hi in spans])
            if case["add"]:
                out += s["dW"].to(f)
        return out
    if op == "combine_grad":
        T, k = case["T"], case["k"]
        out, dg = s["dY_perm"].to(f), torch.zeros((T, k), dtype=f, device="cuda")
        off = s["offsets"].long()
        for j in range(k):
            t = torch.nonzero(s["keep"][:, j])[:, 0]
            r = off[s["topk"][t, j].long()] + s["pos"][t, j].long()
            dy = s["dy"][t].to(f)
            out[r] = s["gates"][t, j, None].to(f) * dy
            dg[t, j] = torch.einsum("td,td->t", dy, s["Y_perm"][r].to(f))
        return {"dY_perm": out, "dgates": dg}
    if op == "ffn_grad":
        sizes, off, _ = _ffn_groups(case)
        spans = [(int(off[i]), int(off[i] + sizes[i])) for i in range(case["E"])]
        return _exact_ffn(s, case, spans)
    return torch.stack([_exact_orthogonalize(g.to(f)) for g in s["G"]])


def _exact_one(x, dy, W1, W3, W2, act):
    """One expert's gradients from the derivatives of erf and of x / (1 + exp(-x))."""
    f = torch.float64
    x, dy, W1, W2 = x.to(f), dy.to(f), W1.to(f), W2.to(f)
    u, dh = x @ W1.T, dy @ W2
    if act == 0:
        phi = torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
        Phi = torch.special.ndtr(u)
        h, du = u * Phi, dh * (Phi + u * phi)
        return du @ W1, du.T @ x, None, dy.T @ h
    v = x @ W3.to(f).T
    g = 1 / (1 + torch.exp(-u))
    silu, slope = u * g, g + u * g * (1 - g)
    du, dv = dh * v * slope, dh * silu
    return du @ W1 + dv @ W3.to(f), du.T @ x, dv.T @ x, dy.T @ (silu * v)


def _exact_ffn(s, case, spans):
    act = case["act"]
    dx, dW = s["dx_perm"].to(torch.float64), []
    for i, (lo, hi) in enumerate(spans):
        W3 = s["W3"][i] if act else None
        r = _exact_one(s["x_perm"][lo:hi], s["dY_perm"][lo:hi], s["W1"][i], W3, s["W2"][i], act)
        dx[lo:hi] = r[0]
        dW.append(r[1:])
    out = [dx] + [None if t[0] is None else torch.stack(t) for t in zip(*dW)]
    if case["n_shared"]:
        rs = [_exact_one(s["x"], s["dy"], s["Ws1"][i], s["Ws3"][i] if act else None, s["Ws2"][i],
                         act) for i in range(case["n_shared"])]
        out.append(sum(r[0] for r in rs))
        out += [None if t[0] is None else torch.stack(t) for t in list(zip(*rs))[1:]]
    return _named(*out)


def _exact_orthogonalize(g):
    """The quintic applied to the singular values, the singular vectors kept."""
    a, b, c = NS_COEFFS
    x = g / (torch.linalg.matrix_norm(g) + NS_EPS)
    for _ in range(NS_STEPS):
        if x.shape[0] <= x.shape[1]:
            q = x @ x.T
            x = a * x + b * (q @ x) + c * (q @ (q @ x))
        else:
            q = x.T @ x
            x = a * x + b * (x @ q) + c * ((x @ q) @ q)
    return x

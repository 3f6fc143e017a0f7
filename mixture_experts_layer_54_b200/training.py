"""Binding of the expert training calls: the grouped products and their
gradients, the gradients of the combine and of the expert FFNs, and the
orthogonalised update.  Argument checks and marshalling only, as in ops.py;
buffers that are not given are allocated with torch.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, replace

import torch

from ._abi import MoeConfig, check, lib
from .ops import DTYPE_BF16, DTYPE_F32, _p, _tdtype, moe_validate

_CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _code(t, what):
    if t.dtype not in _CODES:
        raise ValueError(f"{what} is {t.dtype}: fp32 or bf16 wanted")
    return _CODES[t.dtype]


def _ptrs(*tensors):
    """Device addresses of the tensors (None for None), after ops._p's checks.
    One look at the current device serves the call."""
    dev, out = None, []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        at = t.get_device()
        if at < 0 or not t.is_contiguous():
            _p(t)   # says what is wrong
        if dev is None:
            dev = torch.cuda.current_device()
        if at != dev:
            _p(t)
        out.append(t.data_ptr())
    return out


def _stream():
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _rows(cfg):
    R = lib().moe_perm_rows(ctypes.byref(cfg))
    if R < 0:
        moe_validate(cfg)
    return R


def _is(t, shape, dtype, what):
    """The library reads raw buffers: a wrong shape or type is refused here."""
    if t is None:
        return
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{what} is {t.dtype} {tuple(t.shape)}: "
                         f"{dtype} {tuple(shape)} wanted")


def _fit(specs):
    """_is of every (tensor, shape, dtype, name), without a call each."""
    for t, shape, dtype, what in specs:
        if t is not None and (t.shape != shape or t.dtype is not dtype):
            _is(t, shape, dtype, what)


def _grouped(a, W_shape, width, offsets, rows, what):
    """(code, G, R, N, K) of a grouped product whose tall operand is a."""
    shape = a.shape
    if len(shape) != 2 or len(W_shape) != 3 or shape[1] != width:
        raise ValueError(f"{what} {tuple(shape)} does not fit weights {tuple(W_shape)}")
    G, N, K = W_shape
    _is(offsets, (G + 1,), torch.int32, "offsets")
    if rows is not None:
        _is(rows, (G,), torch.int32, "rows")
    return _code(a, what), G, shape[0], N, K


def _workspace(nbytes, like):
    # new_empty takes half as long as torch.empty with a device
    return like.new_empty(max(nbytes, 256), dtype=torch.uint8)


def moe_grouped_workspace_size(dtype, G: int, R: int, N: int, K: int) -> int:
    """Bytes of the workspace of the three grouped products; 0 for sizes they refuse."""
    return int(lib().moe_grouped_workspace_size(_CODES.get(dtype, -1), int(G), int(R), int(N), int(K)))


_grouped_bytes = 0


def _grouped_ws(sizes, ws, like):
    """(workspace, bytes): the fp32 products do without; one size serves every
    bf16 product (too small a one would be refused)."""
    global _grouped_bytes
    if ws is None:
        if sizes[0] == DTYPE_F32:
            return None, 0
        if not _grouped_bytes:
            _grouped_bytes = lib().moe_grouped_workspace_size(DTYPE_BF16, 1, 1, 8, 8)
        ws = _workspace(_grouped_bytes, like)
    return ws, ws.numel()


def moe_grouped_matmul(x, W, offsets, rows=None, y=None, ws=None):
    """y[r] = W[g] x[r] for the rows r of each group g: x [R, K], W [G, N, K],
    offsets [G + 1] (and rows [G]) int32.  Rows of no group are not written."""
    W_shape = W.shape
    sizes = _grouped(x, W_shape, W_shape[-1], offsets, rows, "x")
    _is(W, W_shape, x.dtype, "W")
    shape = (sizes[2], sizes[3])
    if y is None:
        y = x.new_empty(shape)
    else:
        _is(y, shape, x.dtype, "y")
    ws, nbytes = _grouped_ws(sizes, ws, x)
    check(lib().moe_grouped_matmul(*sizes, *_ptrs(x, W, offsets, rows, y, ws), nbytes,
                                   _stream()), "moe_grouped_matmul")
    return y


def moe_grouped_matmul_dx(dy, W, offsets, rows=None, dx=None, ws=None):
    """Gradient of moe_grouped_matmul by x: dx[r] = W[g]^T dy[r], dy [R, N]."""
    W_shape = W.shape
    sizes = _grouped(dy, W_shape, W_shape[-2], offsets, rows, "dy")
    _is(W, W_shape, dy.dtype, "W")
    shape = (sizes[2], sizes[4])
    if dx is None:
        dx = dy.new_empty(shape)
    else:
        _is(dx, shape, dy.dtype, "dx")
    ws, nbytes = _grouped_ws(sizes, ws, dy)
    check(lib().moe_grouped_matmul_dx(*sizes, *_ptrs(dy, W, offsets, rows, dx, ws), nbytes,
                                      _stream()), "moe_grouped_matmul_dx")
    return dx


def moe_grouped_matmul_dw(dy, x, offsets, rows=None, add=None, dW=None, out_dtype=None, ws=None):
    """Gradient of moe_grouped_matmul by W: dW[g] = (add[g] +) sum of dy[r] x[r]^T
    over the rows r of group g.  dW may be add itself (summing over
    micro-batches); out_dtype defaults to that of add, dW or dy."""
    G = offsets.shape[0] - 1
    if dy.dim() != 2 or x.dim() != 2:
        raise ValueError("dy and x are [R, N] and [R, K]")
    shape = (G, dy.shape[1], x.shape[1])
    sizes = _grouped(dy, shape, shape[1], offsets, rows, "dy")
    _is(x, (sizes[2], shape[2]), dy.dtype, "x")
    if out_dtype is None:
        out_dtype = next((t.dtype for t in (add, dW) if t is not None), dy.dtype)
    if dW is None:
        dW = dy.new_empty(shape, dtype=out_dtype)
    else:
        _is(dW, shape, out_dtype, "dW")
    _is(add, shape, out_dtype, "add")
    ws, nbytes = _grouped_ws(sizes, ws, dy)
    check(lib().moe_grouped_matmul_dw(*sizes, *_ptrs(dy, x, offsets, rows), _code(dW, "dW"),
                                      *_ptrs(add, dW, ws), nbytes, _stream()),
          "moe_grouped_matmul_dw")
    return dW


def moe_combine_backward(cfg: MoeConfig, dy, Y_perm, gates, topk, pos, keep, offsets, dY_perm=None,
                         dgates=None):
    """Gradients of moe_combine: (dY_perm, dgates).  Padding rows of dY_perm are
    not written."""
    T, k, d, dt = cfg.T, cfg.k, cfg.d, _tdtype(cfg)
    R = _rows(cfg)
    rd, tk, f32, i32 = (R, d), (T, k), torch.float32, torch.int32
    _fit(((dy, (T, d), dt, "dy"), (Y_perm, rd, dt, "Y_perm"), (dY_perm, rd, dt, "dY_perm"),
          (gates, tk, f32, "gates"), (dgates, tk, f32, "dgates"), (topk, tk, i32, "topk"),
          (pos, tk, i32, "pos"), (keep, tk, torch.uint8, "keep"),
          (offsets, (cfg.E + 1,), i32, "offsets")))
    if dY_perm is None:
        dY_perm = dy.new_empty(rd)
    if dgates is None:
        dgates = torch.empty_like(gates)
    check(lib().moe_combine_backward(ctypes.byref(cfg), *_ptrs(dy, Y_perm, gates, topk, pos, keep,
                                                               offsets, dY_perm, dgates),
                                     _stream()), "moe_combine_backward")
    return dY_perm, dgates


def moe_ffn_backward_workspace_size(cfg: MoeConfig) -> int:
    return int(lib().moe_ffn_backward_workspace_size(ctypes.byref(cfg)))


@dataclass
class FFNGrads:
    """Gradients of moe_expert_ffn's inputs (None where the layer has none)."""
    dx_perm: torch.Tensor
    dW1: torch.Tensor
    dW3: torch.Tensor | None
    dW2: torch.Tensor
    dx_shared: torch.Tensor | None = None
    dWs1: torch.Tensor | None = None
    dWs3: torch.Tensor | None = None
    dWs2: torch.Tensor | None = None


def moe_expert_ffn_backward(cfg: MoeConfig, x_perm, offsets, kept, dY_perm, W1, W3, W2, x=None,
                            dY_shared=None, Ws1=None, Ws3=None, Ws2=None, dx_perm=None,
                            grads: FFNGrads | None = None, dw_dtype=None, accumulate=False,
                            ws=None) -> FFNGrads:
    """Gradients of moe_expert_ffn, the hidden activations computed again from
    x_perm (and x for the shared experts).  kept [E] are the capacity stage's row
    counts.  `grads` gives the output buffers (dx_perm alone its own); with
    accumulate the weight gradients are added to what they hold."""
    E, d, F, T, S, Fs = cfg.E, cfg.d, cfg.d_ff, cfg.T, cfg.n_shared, cfg.d_ff_shared
    dt = _tdtype(cfg)
    R = _rows(cfg)
    swiglu = cfg.act == 1
    if accumulate and grads is None:
        raise ValueError("accumulate adds to the weight gradients in `grads`")
    if grads is None:
        wt = dt if dw_dtype is None else dw_dtype
        e = lambda *shape, t=wt: x_perm.new_empty(shape, dtype=t)
        grads = FFNGrads(dx_perm=e(R, d, t=dt) if dx_perm is None else dx_perm, dW1=e(E, F, d),
                         dW3=e(E, F, d) if swiglu else None, dW2=e(E, d, F))
        if S:
            grads.dx_shared = e(T, d, t=dt)
            grads.dWs1, grads.dWs2 = e(S, Fs, d), e(S, d, Fs)
            grads.dWs3 = e(S, Fs, d) if swiglu else None
    elif dx_perm is not None:
        grads = replace(grads, dx_perm=dx_perm)   # the caller's stays as it is
    g = grads
    wt = g.dW1.dtype
    if dw_dtype is not None and dw_dtype != wt:
        raise ValueError(f"dw_dtype {dw_dtype} but dW1 is {wt}")
    _fit((
            (x_perm, (R, d), dt, "x_perm"), (dY_perm, (R, d), dt, "dY_perm"),
            (offsets, (E + 1,), torch.int32, "offsets"), (kept, (E,), torch.int32, "kept"),
            (W1, (E, F, d), dt, "W1"), (W3, (E, F, d), dt, "W3"), (W2, (E, d, F), dt, "W2"),
            (x, (T, d), dt, "x"), (dY_shared, (T, d), dt, "dY_shared"),
            (Ws1, (S, Fs, d), dt, "Ws1"), (Ws3, (S, Fs, d), dt, "Ws3"),
            (Ws2, (S, d, Fs), dt, "Ws2"), (g.dx_perm, (R, d), dt, "dx_perm"),
            (g.dW1, (E, F, d), wt, "dW1"), (g.dW3, (E, F, d), wt, "dW3"),
            (g.dW2, (E, d, F), wt, "dW2"), (g.dx_shared, (T, d), dt, "dx_shared"),
            (g.dWs1, (S, Fs, d), wt, "dWs1"), (g.dWs3, (S, Fs, d), wt, "dWs3"),
            (g.dWs2, (S, d, Fs), wt, "dWs2")))
    if ws is None:
        ws = _workspace(moe_ffn_backward_workspace_size(cfg), x_perm)
    check(lib().moe_expert_ffn_backward(
        ctypes.byref(cfg), *_ptrs(x_perm, offsets, kept, dY_perm, W1, W3, W2, x, dY_shared, Ws1,
                                  Ws3, Ws2, g.dx_perm, g.dW1, g.dW3, g.dW2, g.dx_shared, g.dWs1,
                                  g.dWs3, g.dWs2),
        _code(g.dW1, "dW1"), int(bool(accumulate)), *_ptrs(ws), ws.numel(), _stream()),
        "moe_expert_ffn_backward")
    return grads


def moe_orthogonalize_workspace_size(E: int, m: int, n: int, steps: int = 5) -> int:
    return int(lib().moe_orthogonalize_workspace_size(int(E), int(m), int(n), int(steps)))


def moe_orthogonalize(G, steps=5, coeffs=(3.4445, -4.7750, 2.0315), scale=1.0, eps=1e-7, U=None,
                      ws=None):
    """Every update G[e] ([E, m, n], or one [m, n]; fp32 or bf16) with its
    singular values driven towards 1 by `steps` Newton-Schulz steps, times scale,
    as bf16."""
    if G.dim() not in (2, 3):
        raise ValueError(f"G is {tuple(G.shape)}: [E, m, n] or [m, n] wanted")
    E, m, n = G.shape if G.dim() == 3 else (1, *G.shape)
    if U is None:
        U = G.new_empty(G.shape, dtype=torch.bfloat16)
    _is(U, G.shape, torch.bfloat16, "U")
    if len(coeffs) != 3:
        raise ValueError(f"coeffs are a, b, c, not {len(coeffs)} numbers")
    c = (ctypes.c_float * 3)(*coeffs)
    if ws is None:
        ws = _workspace(moe_orthogonalize_workspace_size(E, m, n, steps), G)
    g, u, w = _ptrs(G, U, ws)
    check(lib().moe_orthogonalize(_code(G, "G"), E, m, n, g, int(steps), c, float(eps),
                                  float(scale), u, w, ws.numel(), _stream()),
          "moe_orthogonalize")
    return U


def moe_training_status() -> int:
    """0, or MOE_ERR_DEVICE_TIMEOUT when a bounded wait of any training call has run
    out on the current device since the last clear (also of calls that made their
    own workspace).  Synchronises the current stream."""
    st = ctypes.c_int32()
    check(lib().moe_training_status(ctypes.byref(st), _stream()), "moe_training_status")
    return int(st.value)


def moe_clear_training_status():
    check(lib().moe_clear_training_status(_stream()), "moe_clear_training_status")


def moe_probe_training_timeout(timeout_ns: int):
    """Diagnostic: one bounded wait that must run out and set the status."""
    check(lib().moe_probe_training_timeout(int(timeout_ns), _stream()),
          "moe_probe_training_timeout")


__all__ = ["moe_grouped_workspace_size", "moe_grouped_matmul", "moe_grouped_matmul_dx",
           "moe_grouped_matmul_dw", "moe_combine_backward", "moe_expert_ffn_backward",
           "moe_ffn_backward_workspace_size", "FFNGrads", "moe_orthogonalize",
           "moe_orthogonalize_workspace_size", "moe_training_status",
           "moe_clear_training_status", "moe_probe_training_timeout"]

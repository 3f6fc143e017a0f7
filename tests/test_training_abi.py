"""Refusals of the expert training calls: every bad argument returns its status
before anything is launched, and the binding refuses wrong shapes and types."""
import ctypes

import pytest
import torch

import mixture_experts_layer_54_b200 as moe
from mixture_experts_layer_54_b200 import _abi, training

P = ctypes.c_void_p(4096)      # aligned, never dereferenced: the checks fail first
ODD = ctypes.c_void_p(4096 + 2)
F32, BF16 = 0, 1


def rows_args(dtype=BF16, G=2, R=10, N=64, K=32, x=P, W=P, off=P, rows=None, y=P, ws=P, nb=1 << 30):
    return dtype, G, R, N, K, x, W, off, rows, y, ws, nb, None


@pytest.mark.parametrize("call", ["moe_grouped_matmul", "moe_grouped_matmul_dx"])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), _abi.MOE_ERR_DTYPE), (dict(G=0), _abi.MOE_ERR_SHAPE),
    (dict(G=257), _abi.MOE_ERR_SHAPE), (dict(R=-1), _abi.MOE_ERR_SHAPE),
    (dict(R=1 << 31), _abi.MOE_ERR_SHAPE), (dict(N=0), _abi.MOE_ERR_SHAPE),
    (dict(N=(1 << 20) + 8), _abi.MOE_ERR_SHAPE), (dict(K=1 << 21), _abi.MOE_ERR_SHAPE),
    (dict(N=60), _abi.MOE_ERR_SHAPE), (dict(K=33), _abi.MOE_ERR_SHAPE),
    (dict(x=None), _abi.MOE_ERR_NULL), (dict(W=None), _abi.MOE_ERR_NULL),
    (dict(off=None), _abi.MOE_ERR_NULL), (dict(y=None), _abi.MOE_ERR_NULL),
    (dict(ws=None), _abi.MOE_ERR_NULL), (dict(x=ODD), _abi.MOE_ERR_ALIGN),
    (dict(W=ODD), _abi.MOE_ERR_ALIGN), (dict(y=ODD), _abi.MOE_ERR_ALIGN),
    (dict(ws=ODD), _abi.MOE_ERR_ALIGN), (dict(nb=255), _abi.MOE_ERR_WORKSPACE)])
def test_grouped_products_check_their_arguments(call, kw, status):
    assert getattr(moe.lib(), call)(*rows_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32, out=BF16), _abi.MOE_ERR_DTYPE), (dict(out=2), _abi.MOE_ERR_DTYPE),
    (dict(K=12), _abi.MOE_ERR_SHAPE), (dict(dW=None), _abi.MOE_ERR_NULL),
    (dict(dy=None), _abi.MOE_ERR_NULL), (dict(add=ODD), _abi.MOE_ERR_ALIGN),
    (dict(dW=ODD), _abi.MOE_ERR_ALIGN), (dict(nb=0), _abi.MOE_ERR_WORKSPACE)])
def test_weight_gradient_checks_its_arguments(kw, status):
    a = dict(dtype=BF16, G=2, R=10, N=64, K=32, dy=P, x=P, off=P, rows=None, out=F32, add=None,
             dW=P, ws=P, nb=1 << 30)
    a.update(kw)
    assert moe.lib().moe_grouped_matmul_dw(*a.values(), None) == status


def test_fp32_products_take_no_workspace():
    """Only bf16 needs one: with none, the fp32 call gets past the check (and, no
    rows, launches nothing)."""
    L = moe.lib()
    assert L.moe_grouped_matmul(*rows_args(dtype=F32, R=0, ws=None, nb=0)) == _abi.MOE_OK
    assert L.moe_grouped_matmul_dx(*rows_args(dtype=F32, R=0, ws=None, nb=0)) == _abi.MOE_OK
    assert L.moe_grouped_matmul(*rows_args(dtype=F32, R=0, ws=P, nb=8)) == _abi.MOE_ERR_WORKSPACE


def test_workspace_sizes():
    L = moe.lib()
    assert L.moe_grouped_workspace_size(BF16, 4, 100, 64, 64) >= 256
    assert L.moe_grouped_workspace_size(BF16, 4, 100, 60, 64) == 0
    cfg = moe.moe_config(T=100, d=128, E=4, k=2, d_ff=192, act=1, dtype=1, cf=1.5, n_shared=2,
                         d_ff_shared=64)
    R = moe.moe_perm_rows(cfg)
    assert moe.moe_ffn_backward_workspace_size(cfg) >= 3 * 2 * (R * 192 + 2 * 100 * 64)
    assert moe.moe_ffn_backward_workspace_size(moe.moe_config(cfg, d_ff=100)) == 0
    assert moe.moe_orthogonalize_workspace_size(3, 100, 50) >= 256
    assert moe.moe_orthogonalize_workspace_size(3, 500, 200) >= 3 * (8 * 500 * 200 + 4 * 200 * 200)
    for bad in ((0, 8, 8, 5), (1025, 8, 8, 5), (1, 0, 8, 5), (1, 8, 0, 5), (1, 8, 8, 0),
                (1, 8, 8, 33), (1, (1 << 20) + 1, 8, 5)):
        assert moe.moe_orthogonalize_workspace_size(*bad) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), _abi.MOE_ERR_DTYPE), (dict(m=0), _abi.MOE_ERR_SHAPE),
    (dict(steps=0), _abi.MOE_ERR_SHAPE), (dict(G=None), _abi.MOE_ERR_NULL),
    (dict(U=None), _abi.MOE_ERR_NULL), (dict(eps=-1.0), _abi.MOE_ERR_SHAPE),
    (dict(eps=float("nan")), _abi.MOE_ERR_SHAPE), (dict(scale=float("inf")), _abi.MOE_ERR_SHAPE),
    (dict(coeffs=(float("nan"), 0, 0)), _abi.MOE_ERR_SHAPE),
    (dict(U=ctypes.c_void_p(4097)), _abi.MOE_ERR_ALIGN), (dict(nb=256), _abi.MOE_ERR_WORKSPACE)])
def test_orthogonalize_checks_its_arguments(kw, status):
    a = dict(dtype=BF16, E=2, m=160, n=240, G=P, steps=5, coeffs=(3.0, -4.0, 2.0), eps=1e-7,
             scale=1.0, U=P, ws=P, nb=1 << 30)
    a.update(kw)
    a["coeffs"] = (ctypes.c_float * 3)(*a["coeffs"])
    assert moe.lib().moe_orthogonalize(*a.values(), None) == status


def ffn_args(cfg, **kw):
    names = ("x_perm offsets kept dY W1 W3 W2 x dy Ws1 Ws3 Ws2 dx dW1 dW3 dW2 dxs dWs1 dWs3 "
             "dWs2").split()
    a = {n: P for n in names}
    a.update(out=BF16, acc=0, ws=P, nb=1 << 40)
    a.update(kw)
    return (ctypes.byref(cfg), *a.values(), None)


def test_ffn_backward_checks_its_arguments():
    L = moe.lib()
    cfg = moe.moe_config(T=64, d=128, E=8, k=2, d_ff=128, act=1, dtype=1, cf=1.0, n_shared=1,
                         d_ff_shared=64)
    call = lambda c=cfg, **kw: L.moe_expert_ffn_backward(*ffn_args(c, **kw))
    for name in ("x_perm", "offsets", "kept", "dY", "W1", "W3", "W2", "x", "dy", "Ws1", "Ws3",
                 "Ws2", "dx", "dW1", "dW3", "dW2", "dxs", "dWs1", "dWs3", "dWs2", "ws"):
        assert call(**{name: None}) == _abi.MOE_ERR_NULL, name
    for name in ("x_perm", "W2", "dWs1"):
        assert call(**{name: ODD}) == _abi.MOE_ERR_ALIGN
    need = moe.moe_ffn_backward_workspace_size(cfg)
    assert call(nb=need - 1) == _abi.MOE_ERR_WORKSPACE
    assert call(out=5) == _abi.MOE_ERR_DTYPE
    assert call(moe.moe_config(cfg, dtype=0), out=BF16) == _abi.MOE_ERR_DTYPE
    assert call(moe.moe_config(cfg, n_shared=65)) == _abi.MOE_ERR_SHAPE
    assert call(moe.moe_config(cfg, cf=0.5)) == _abi.MOE_ERR_CAPACITY_FACTOR


def test_combine_backward_checks_its_arguments():
    L = moe.lib()
    cfg = moe.moe_config(T=64, d=128, E=8, k=2, d_ff=128, act=1, dtype=1, cf=1.0)
    for i in range(9):
        a = [P] * 9
        a[i] = None
        assert L.moe_combine_backward(ctypes.byref(cfg), *a, None) == _abi.MOE_ERR_NULL
    assert L.moe_combine_backward(ctypes.byref(cfg), ODD, *[P] * 8, None) == _abi.MOE_ERR_ALIGN
    none = moe.moe_config(cfg, T=0)
    assert L.moe_combine_backward(ctypes.byref(none), *[None] * 9, None) == _abi.MOE_OK


def test_binding_refuses_wrong_shapes_types_and_places():
    bf, i32 = torch.bfloat16, torch.int32
    x, W = torch.zeros((6, 32), dtype=bf), torch.zeros((2, 64, 32), dtype=bf)
    off = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_matmul(x, W, off, ws=torch.zeros(256, dtype=torch.uint8))
    for bad in (dict(x=x.half()), dict(x=x[:, :24].contiguous()), dict(W=W.float()),
                dict(offsets=off.long()), dict(offsets=torch.zeros(4, dtype=i32)),
                dict(rows=torch.zeros(3, dtype=i32)), dict(y=torch.zeros((6, 32), dtype=bf)),
                dict(x=x[0])):
        with pytest.raises(ValueError):
            moe.moe_grouped_matmul(**(dict(x=x, W=W, offsets=off) | bad))
    dy = torch.zeros((6, 64), dtype=bf)
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_dx(x, W, off)
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_dw(dy, x[:5], off)
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_dw(dy, x, off, add=torch.zeros((2, 64, 32)),
                                  out_dtype=bf)
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(torch.zeros(5))
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(torch.zeros((5, 4), dtype=torch.float64))
    cfg = moe.moe_config(T=4, d=64, E=2, k=1, d_ff=64, act=0, dtype=1, cf=1.0)
    with pytest.raises(ValueError, match="accumulate"):
        moe.moe_expert_ffn_backward(cfg, x, off, off, x, W, None, W, accumulate=True)
    with pytest.raises(ValueError, match="x_perm"):
        moe.moe_expert_ffn_backward(cfg, x, off, off, x, W, None, W)
    with pytest.raises(ValueError, match="dy"):
        moe.moe_combine_backward(cfg, x, x, x, x, x, x, off)


def test_package_exports_every_training_binding():
    assert set(training.__all__) <= set(moe.__all__)


@pytest.mark.parametrize("coeffs,steps", [
    ((2.85, 0.0, 0.0), 2), ((2.7, 0.0, 0.0), 3), ((1.0, 31.0, 0.0), 1), ((32.0, -31.5, 0.0), 1),
    ((-33.0, 0.0, 0.0), 1), ((3.0, -4.0, 2.0), 5), ((0.0, 0.0, 3.0), 2), ((0.5, 40.0, -40.0), 2),
    ((1e30, 1.0, 1e-30), 2), ((1.0, -3e38, 3e38), 1)])
def test_orthogonalize_refuses_steps_that_leave_fp16(coeffs, steps):
    """(E, m, n) of the form of many launches and of the one-launch form."""
    if torch.cuda.is_available():
        pytest.skip("pointers of no memory: without a device nothing can be launched with them")
    for m, n in ((160, 240), (16, 16)):
        c = (ctypes.c_float * 3)(*coeffs)
        status = moe.lib().moe_orthogonalize(BF16, 2, m, n, P, steps, c, 1e-7, 1.0, P, P, 1 << 30, None)
        assert status == _abi.MOE_ERR_SHAPE


def test_grouped_workspace_size_of_the_binding():
    size = moe.moe_grouped_workspace_size
    assert size(torch.bfloat16, 4, 100, 64, 64) == moe.lib().moe_grouped_workspace_size(BF16, 4, 100, 64, 64)
    assert size(torch.bfloat16, 4, 100, 60, 64) == 0 and size(torch.float32, 4, 100, 60, 64) >= 256
    assert size(torch.float16, 4, 100, 64, 64) == 0


def test_training_status_checks_its_arguments():
    assert moe.lib().moe_training_status(None, None) == _abi.MOE_ERR_NULL
    assert moe.lib().moe_probe_training_timeout(2_000_000_001, None) == _abi.MOE_ERR_SHAPE


def test_ffn_backward_leaves_the_callers_gradients_alone():
    """dx_perm beside `grads` is used for this call; the caller's object keeps its own."""
    cfg = moe.moe_config(T=4, d=64, E=2, k=1, d_ff=64, act=0, dtype=1, cf=1.0)
    R, bf = moe.moe_perm_rows(cfg), torch.bfloat16
    x, W = torch.zeros((R, 64), dtype=bf), torch.zeros((2, 64, 64), dtype=bf)
    off, kept = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    mine = torch.zeros((R, 64), dtype=bf)
    grads = moe.FFNGrads(dx_perm=mine, dW1=W, dW3=None, dW2=W)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_expert_ffn_backward(cfg, x, off, kept, x, W, None, W, grads=grads,
                                    dx_perm=torch.zeros_like(x), ws=torch.zeros(256, dtype=torch.uint8))
    assert grads.dx_perm is mine

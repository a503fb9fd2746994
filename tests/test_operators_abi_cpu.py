"""Argument checks of the operators around the layer, all made on the host
before any device call (no compute here)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def test_norm_forward_refusals(m):
    f = m.lib.fp8_add_rmsnorm_quant_1x128
    ok = dict(x=16, ld_x=256, r=None, ld_r=0, dt=0, w=None, eps=1e-6, rows=4, cols=256, h=None, y=None, q=16, s=16,
              rstd=None, mode=0)

    def call(**kw):
        a = {**ok, **kw}
        return f(*[a[k] for k in ok], None)

    assert call() == m.MOE_ERR_NO_DEVICE
    assert call(rows=0, x=None, q=None, s=None) == m.MOE_OK
    assert call(cols=200, ld_x=200) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(cols=32768 + 128, ld_x=1 << 16) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(rows=1 << 31) == m.MOE_ERR_UNSUPPORTED_SHAPE
    for bad in (dict(ld_x=128), dict(ld_x=257), dict(rows=-1), dict(cols=0), dict(dt=2), dict(mode=2), dict(eps=0.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(q=None), dict(s=None), dict(x=24),
                dict(s=18), dict(y=24), dict(w=20), dict(rstd=18),
                dict(r=16, ld_r=256), dict(r=16, ld_r=128, h=32), dict(r=16, ld_r=260, h=32),
                dict(r=16, ld_r=264, h=16), dict(h=16, ld_x=264)):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert call(r=16, ld_r=256, h=16) == m.MOE_ERR_NO_DEVICE


def test_norm_backward_refusals(m):
    f = m.lib.add_rmsnorm_backward
    need = m.lib.add_rmsnorm_backward_workspace_size(4, 256)
    assert need >= 256 and m.lib.add_rmsnorm_backward_workspace_size(4, 100) == 0
    ok = dict(dy=16, dyt=1, h=32, dres=None, dt=0, w=None, rstd=16, rows=4, cols=256, dx=48, dxt=0, dw=16, ws=256,
              n=need)

    def call(**kw):
        a = {**ok, **kw}
        return f(*[a[k] for k in ok], None)

    assert call() == m.MOE_ERR_NO_DEVICE
    assert call(n=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(dw=None, ws=None, n=0) == m.MOE_ERR_NO_DEVICE
    assert call(rows=0, dw=None) == m.MOE_OK
    assert call(cols=130) == m.MOE_ERR_UNSUPPORTED_SHAPE
    for bad in (dict(dyt=5), dict(dt=-1), dict(dxt=2), dict(rows=-1), dict(dy=None), dict(h=None), dict(rstd=None),
                dict(dx=None), dict(ws=None), dict(ws=128), dict(dx=24), dict(dres=24), dict(dw=18),
                dict(dx=16), dict(dx=32, dxt=1)):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert call(dx=16, dxt=1) == m.MOE_ERR_NO_DEVICE and call(dx=32) == m.MOE_ERR_NO_DEVICE


def test_balance_refusals(m):
    cfg = m.config(512, 256, 16, 4)
    need = m.lib.moe_balance_loss_workspace_size(C.byref(cfg), 64, 3)
    assert need >= 256
    ok = dict(cfg=C.byref(cfg), z=16, ns=2, idx=16, T=64, off=16, n=3, alpha=1e-4, loss=16, counts=16, ws=256, wb=need,
              err=16)

    def call(**kw):
        a = {**ok, **kw}
        return m.lib.moe_balance_loss(*[a[k] for k in ok], None)

    assert call() == m.MOE_ERR_NO_DEVICE
    assert call(n=0, off=None, loss=None, counts=None, ws=None) == m.MOE_OK
    assert call(wb=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(cfg=None), dict(ns=0), dict(ns=1025), dict(T=-1), dict(T=(1 << 20) + 1), dict(n=-1),
                dict(alpha=float("nan")), dict(z=None), dict(z=20), dict(idx=None), dict(off=None), dict(loss=18),
                dict(counts=None), dict(ws=128), dict(err=None)):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad


def test_router_backward_refusals(m):
    cfg = m.config(512, 256, 16, 4)
    need = m.lib.moe_router_backward_workspace_size(C.byref(cfg), 64)
    assert need >= 3 * 64 * 64 * 2
    B = m._binding.MoeBalanceGrad
    bal = B(16, 3, 1e-4, 16, None)
    ok = dict(cfg=C.byref(cfg), z=16, ns=1, idx=16, T=64, dgate=16, bal=C.byref(bal), x=16, wr=16, dz=16, dx=16, acc=0,
              dwr=16, ws=256, wb=need, err=16)

    def call(**kw):
        a = {**ok, **kw}
        return m.lib.moe_router_backward(*[a[k] for k in ok], None)

    assert call() == m.MOE_ERR_NO_DEVICE
    assert call(dx=None, dwr=None, ws=None, wb=0, x=None, wr=None) == m.MOE_ERR_NO_DEVICE
    assert call(T=0, dwr=None) == m.MOE_OK
    assert call(wb=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(cfg=None), dict(ns=0), dict(T=-1), dict(x=None), dict(wr=None), dict(z=None), dict(idx=None),
                dict(ws=None), dict(ws=128), dict(err=None), dict(dx=20), dict(dwr=20), dict(x=20), dict(wr=24),
                dict(dz=18), dict(dgate=18), dict(bal=C.byref(B(None, 3, 1e-4, 16, None))),
                dict(bal=C.byref(B(16, 3, 1e-4, None, None))), dict(bal=C.byref(B(16, -1, 1e-4, 16, None))),
                dict(bal=C.byref(B(16, 3, float("nan"), 16, None))), dict(bal=C.byref(B(16, 3, 1e-4, 16, 18)))):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert m.moe_router_splits(cfg, 64) >= 1
    with pytest.raises(m.MoeError):
        m.moe_router_splits(cfg, -1)


def test_bindings_refuse_host_tensors(m):
    cfg = m.config(512, 256, 16, 4)
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(m.MoeError, match="CUDA device"):
        m.fp8_add_rmsnorm_quant_1x128(x)
    with pytest.raises(m.MoeError):
        m.add_rmsnorm_backward(x, x, torch.zeros(2))
    with pytest.raises(m.MoeError):
        m.moe_balance_loss(cfg, torch.zeros((1, 2, 16)), torch.zeros((2, 4), dtype=torch.int32),
                           torch.zeros(2, dtype=torch.int32))
    with pytest.raises(m.MoeError):
        m.moe_router_backward(cfg, torch.zeros((1, 2, 16)), torch.zeros((2, 4), dtype=torch.int32), dlogits=True)


def test_block_refusals(m):
    cfg = m.config(512, 256, 16, 4)
    w = m._binding.MoeWeights(16, 16, 16, 16, 16)
    need = m.moe_workspace_size(cfg, 64)
    ok = dict(cfg=C.byref(cfg), w=C.byref(w), bias=16, nw=None, eps=1e-6, x=16, r=None, T=64, h=None, y=16, rstd=None,
              out=16, od=0, idx=None, cnt=None, ws=256, wb=need, err=16)

    def fwd(**kw):
        a = {**ok, **kw}
        return m.lib.moe_block_forward(*[a[k] for k in ok], None)

    assert fwd() == m.MOE_ERR_NO_DEVICE and fwd(r=16, h=32) == m.MOE_ERR_NO_DEVICE
    assert fwd(T=0) == m.MOE_OK
    assert fwd(wb=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(cfg=None), dict(w=None), dict(bias=None), dict(eps=0.0), dict(x=None), dict(y=None), dict(r=16),
                dict(T=-1), dict(od=3), dict(out=None), dict(ws=128), dict(err=None), dict(nw=20), dict(y=24),
                dict(rstd=18), dict(h=24)):
        assert fwd(**bad) == m.MOE_ERR_INVALID_ARG, bad

    need_b = m.lib.moe_block_backward_workspace_size(C.byref(cfg), 64)
    assert need_b > m.lib.moe_backward_workspace_size(C.byref(cfg), 64)
    okb = dict(cfg=C.byref(cfg), w=C.byref(w), a=16, b=16, c=16, d=16, nw=None, h=16, y=16, rstd=16, dout=16, T=64,
               bal=None, dx=16, dxt=0, dn=None, dwr=16, dW13=16, dW2=16, f=256, fb=need, ws=256, wb=need_b, err=16)

    def bwd(**kw):
        a = {**okb, **kw}
        return m.lib.moe_block_backward(*[a[k] for k in okb], None)

    assert bwd() == m.MOE_ERR_NO_DEVICE
    assert bwd(wb=need_b - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL and bwd(fb=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    p2 = m.config(512, 256, 16, 4, scale_mode=m.MOE_SCALE_POW2)
    assert bwd(cfg=C.byref(p2)) == m.MOE_ERR_NOT_IMPLEMENTED
    bal = m._binding.MoeBalanceGrad(16, 2, 1e-4, None, None)
    for bad in (dict(T=0), dict(h=None), dict(y=None), dict(rstd=None), dict(dout=None), dict(dx=None), dict(dwr=None),
                dict(dW13=None), dict(f=None), dict(ws=128), dict(err=None), dict(dxt=2), dict(dx=24), dict(nw=20),
                dict(bal=C.byref(bal))):
        assert bwd(**bad) == m.MOE_ERR_INVALID_ARG, bad


def test_block_backward_in_place_refusals(m):
    """dx may take the place of dout, h or y in bf16 alone: FP32 rows are wider."""
    cfg = m.config(512, 256, 16, 4)
    w = m._binding.MoeWeights(16, 16, 16, 16, 16)
    need = m.moe_workspace_size(cfg, 64)
    need_b = m.lib.moe_block_backward_workspace_size(C.byref(cfg), 64)

    def bwd(dx, dxt):
        h, y, dout = 32, 48, 64
        return m.lib.moe_block_backward(C.byref(cfg), C.byref(w), 16, 16, 16, 16, None, h, y, 16, dout, 64, None, dx,
                                        dxt, None, 16, 16, 16, 256, need, 256, need_b, 16, None)

    for dx in (32, 48, 64):
        assert bwd(dx, 1) == m.MOE_ERR_INVALID_ARG and bwd(dx, 0) == m.MOE_ERR_NO_DEVICE
    assert bwd(80, 1) == m.MOE_ERR_NO_DEVICE

"""Operators around the layer (residual + RMS norm + FP8 quantization, its
backward, the balance loss of packed sequences, the router's backward) against
the 64-bit oracle.

Tolerances count roundings: U = 2^-24 is half a step of FP32 relative to the
value, a sum of n FP32 terms in a chain of depth d is off by at most
d U sum|terms| (first order), a result stored as bf16 by 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from _moe_util import guarded_empty
from oracle import block as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def f64(t):
    return t.detach().cpu().double().numpy()


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------- norm
# a thread adds up to 4 chunks of 8 squares, then 5 butterfly steps, then up to 32 warps; mean, + eps, sqrt, 1/x
RSTD_TOL = ((32 + 5 + 32) / 2 + 4) * U
Y_TOL = RSTD_TOL + 2 * U  # two products


def norm_inputs(T, H, dtype, resid, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, ld or H), generator=g).to(dtype)
    r = (torch.randn((T, ld or H), generator=g) * 2).to(dtype) if resid else None
    w = 1 + 0.2 * torch.randn((H,), generator=g)
    return x.cuda()[:, :H], None if r is None else r.cuda()[:, :H], w.cuda()


def check_norm(m, x, resid, w, pow2, out):
    h, y, q, s, rstd = out
    T, H = x.shape
    href = x.float() if resid is None else (x.float() + resid.float()).to(x.dtype).float()
    assert torch.equal(h.float(), href)
    yr, rr = O.rmsnorm(f64(href), None if w is None else f64(w), EPS)
    assert (np.abs(f64(rstd) - rr) <= RSTD_TOL * rr).all()
    assert (np.abs(f64(y) - yr) <= (half(torch.bfloat16) + 2 * Y_TOL) * np.abs(yr) + 2.0 ** -133).all()
    amax, sg = O.tile_amax(yr), f64(s)
    if pow2:
        nz = amax > 0
        assert (sg[~nz] == 0).all() and (np.log2(sg[nz]) % 1 == 0).all()
        assert (448 * sg[nz] >= amax[nz] * (1 - Y_TOL)).all() and (224 * sg[nz] < amax[nz] * (1 + Y_TOL)).all()
    else:
        assert (np.abs(sg - amax / 448) <= (Y_TOL + U) * amax / 448 + 2.0 ** -150).all()
    u = np.where(np.repeat(sg, 128, 1) > 0, yr / np.where(np.repeat(sg, 128, 1) > 0, np.repeat(sg, 128, 1), 1), 0)
    codes = q.view(torch.float8_e4m3fn).float().cpu().double().numpy()
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -6))), -6) - 3)
    # the nearest code of a value within (Y_TOL + division) of y / S
    assert (np.abs(codes - np.clip(u, -448, 448)) <= step / 2 + (Y_TOL + 2 * U) * np.abs(u)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (3, 384), (37, 512), (64, 7168), (5, 1152), (2, 8320), (2, 32768),
                                 (513, 1024), (1300, 7168), (700, 16384), (5001, 128)])
def test_norm_forward(m, T, H, dtype):
    for k, (resid, pow2, weight) in enumerate([(True, False, True), (False, True, True), (True, True, False)]):
        x, r, w = norm_inputs(T, H, dtype, resid, T + H + k)
        w = w if weight else None
        check_norm(m, x, r, w, pow2, m.fp8_add_rmsnorm_quant_1x128(x, r, w, EPS, pow2=pow2))


def test_norm_forward_strided_in_place_and_guarded(m):
    T, H = 19, 640
    x, r, w = norm_inputs(T, H, torch.bfloat16, True, 3, ld=H + 72)
    bufs = [guarded_empty((T, H), torch.bfloat16), guarded_empty((T, H), torch.bfloat16),
            guarded_empty((T, H), torch.uint8), guarded_empty((T, H // 128), torch.float32),
            guarded_empty((T,), torch.float32)]
    h, y, q, s, rstd = (b[0] for b in bufs)
    out = m.fp8_add_rmsnorm_quant_1x128(x, r, w, EPS, h=h, y=y, q=q, scales=s, rstd=rstd)
    check_norm(m, x, r, w, False, out)
    for _, check in bufs:
        check()
    # h in the place of the residual stream
    r2 = r.contiguous().clone()
    out2 = m.fp8_add_rmsnorm_quant_1x128(x, r2, w, EPS, h=r2)
    assert out2[0].data_ptr() == r2.data_ptr()
    for a, b in zip(out, out2):
        assert torch.equal(a, b)


def test_norm_sixteen_byte_aligned_buffers(m):
    """Tensors that start 16 bytes into a 32-byte sector, and enough rows for every CTA to take several."""
    T, H = 2500, 256

    def off(dtype, src=None):
        n = 16 // torch.empty((), dtype=dtype).element_size()
        t = torch.empty(T * H + n, dtype=dtype, device="cuda")[n:].view(T, H)
        assert t.data_ptr() % 32 == 16
        return t if src is None else t.copy_(src)

    for dtype in (torch.bfloat16, torch.float32):
        x, r, w = norm_inputs(T, H, dtype, True, 11)
        h, y = off(dtype), off(torch.bfloat16)
        out = m.fp8_add_rmsnorm_quant_1x128(off(dtype, x), off(dtype, r), w, EPS, h=h, y=y)
        check_norm(m, x, r, w, False, out)
        dy = torch.randn((T, H), generator=torch.Generator().manual_seed(1)).cuda()
        want = m.add_rmsnorm_backward(dy, h.clone(), out[4], w, dres=r, dx_dtype=torch.float32)
        got = m.add_rmsnorm_backward(off(torch.float32, dy), h, out[4], w, dres=off(dtype, r), dx=off(torch.float32))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_forward_zero_and_nonfinite_rows(m):
    x, _, w = norm_inputs(4, 512, torch.bfloat16, False, 5)
    x = x.contiguous()
    x[1] = 0
    x[2, 200] = float("nan")
    x[3, 300] = float("inf")
    _, y, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, None, w, EPS)
    assert (y[1] == 0).all() and (q[1] == 0).all() and (s[1] == 0).all()
    assert rstd[1].item() == pytest.approx(EPS ** -0.5, rel=4 * U)
    # a NaN reaches the whole row; an infinity makes rstd 0, and NaN in its own tile only
    assert torch.isnan(s[2]).all() and torch.isnan(y[2]).all()
    assert torch.isnan(q[2].view(torch.float8_e4m3fn).float()).all()
    assert torch.isnan(s[3]).tolist() == [False, False, True, False] and rstd[3] == 0
    assert torch.isnan(y[3, 300]) and torch.isnan(q[3, 256:384].view(torch.float8_e4m3fn).float()).all()
    check_norm(m, x[:1], None, w, False, m.fp8_add_rmsnorm_quant_1x128(x[:1], None, w, EPS))


@pytest.mark.parametrize("dy_t,h_t,dx_t", [(a, b, c) for a in (torch.bfloat16, torch.float32)
                                           for b in (torch.bfloat16, torch.float32)
                                           for c in (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,H", [(1, 128), (9, 384), (300, 7168), (1300, 512), (3, 32768), (2, 8320), (310, 12288), (5000, 128)])
def test_norm_backward(m, T, H, dy_t, h_t, dx_t):
    g = torch.Generator().manual_seed(T + H)
    h = (torch.randn((T, H), generator=g) * 2).to(h_t).cuda()
    dy = torch.randn((T, H), generator=g).to(dy_t).cuda()
    dres = torch.randn((T, H), generator=g).to(h_t).cuda() if T != 9 else None
    w = (1 + 0.2 * torch.randn((H,), generator=g)).cuda() if T != 3 else None
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    (dx, cdx), (dw, cdw) = guarded_empty((T, H), dx_t), guarded_empty((H,), torch.float32)
    m.add_rmsnorm_backward(dy, h, rstd, w, dres=dres, dx=dx, dw=dw)
    cdx(), cdw()
    n = f64(h) * f64(rstd)[:, None]
    gg = f64(dy) * (1 if w is None else f64(w))
    ref, dwr = O.rmsnorm_backward(f64(dy), f64(h), f64(rstd), None if w is None else f64(w),
                                  None if dres is None else f64(dres))
    # n, g: one rounding each; the mean: a chain of 32 + 5 + 32 of products (3 roundings); 3 more to the result
    mag = (0 if dres is None else np.abs(f64(dres))) + f64(rstd)[:, None] * (
        np.abs(gg) + np.abs(n) * np.abs(gg * n).mean(1, keepdims=True))
    assert (np.abs(f64(dx) - ref) <= (69 + 8) * U * mag + half(dx_t) * np.abs(ref) + 2.0 ** -133).all()
    # dw: at most T rows in a chain, then 8 row groups, the CTAs (at most 2 per SM) in 32 chains, 32 more; 2 products
    depth = T + 8 + 40 + 32 + 2
    assert (np.abs(f64(dw) - dwr) <= depth * U * np.abs(f64(dy) * n).sum(0)).all()
    again = m.add_rmsnorm_backward(dy, h, rstd, w, dres=dres, dx_dtype=dx_t)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_norm_backward_in_place_and_empty(m):
    T, H = 33, 256
    g = torch.Generator().manual_seed(0)
    h, dres = (torch.randn((T, H), generator=g).cuda() for _ in range(2))
    dy = torch.randn((T, H), generator=g).cuda()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    want, dw = m.add_rmsnorm_backward(dy, h, rstd, dres=dres)
    for t in (dy, h, dres):
        a = dict(dy=dy, h=h, dres=dres)
        name = [k for k, v in a.items() if v is t][0]
        a[name] = t.clone()
        got, dw2 = m.add_rmsnorm_backward(a["dy"], a["h"], rstd, dres=a["dres"], dx=a[name])
        assert torch.equal(got, want) and torch.equal(dw, dw2)
    e = torch.empty((0, H), device="cuda")
    dw = torch.full((H,), 7.0, device="cuda")
    m.add_rmsnorm_backward(e, e, torch.empty(0, device="cuda"), dw=dw)
    assert (dw == 0).all()
    out = m.fp8_add_rmsnorm_quant_1x128(e)
    assert out[1].shape == (0, H)


# --------------------------------------------------------- balance, router
def router_inputs(T, Nr, Kr, S, seed, std=1.7):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((S, T, Nr), generator=g) * std / S ** 0.5
    idx = logits.sum(0).topk(Kr, dim=1).indices.to(torch.int32) if T else torch.empty((0, Kr), dtype=torch.int32)
    return logits, idx


def z_tol(logits):
    """Relative error of s and of 1 - s: the splits' FP32 sum, expf (2 ulp), 1 + q, 1/x, one product."""
    zabs = logits.abs().sum(0).max().item() if logits.numel() else 0.0
    return (logits.shape[0] * zabs + 2 * 2 + 3) * U


CASES = [  # T, Nr, Kr, S, offsets
    (1, 16, 4, 1, [0, 1]),
    (40, 16, 4, 8, [0, 7, 7, 8, 31]),
    (300, 256, 8, 3, [0, 300]),
    (700, 100, 5, 2, [3, 100, 101, 101, 640]),
    (2500, 256, 8, 1, [0, 2000, 2001, 2400]),
    (97, 1, 1, 1, [0, 50, 97]),
    (130, 33, 16, 2, [0, 0, 130, 130]),
    (64, 256, 8, 1, [10, 10]),
]


@pytest.mark.parametrize("T,Nr,Kr,S,off", CASES)
def test_balance_loss_and_gradient(m, T, Nr, Kr, S, off):
    logits, idx = router_inputs(T, Nr, Kr, S, T)
    z = logits.double().sum(0).numpy()
    cfg = m.config(128, 128, Nr, Kr)
    err = m.new_err_flag()
    offd = torch.tensor(off, dtype=torch.int32).cuda()
    n_seq = len(off) - 1
    (loss, cl), (counts, cc) = guarded_empty((n_seq,), torch.float32), guarded_empty((n_seq, Nr), torch.int32)
    m.moe_balance_loss(cfg, logits.cuda(), idx.cuda(), offd, alpha=0.3, loss=loss, counts=counts, err=err)
    cl(), cc()
    lr, cr = O.balance_loss(z, idx.numpy().astype(np.int64), off, 0.3)
    assert np.array_equal(counts.cpu().numpy(), cr)
    # all terms positive: 8 + 5 terms of sum s, a token chain (at most T/8 in a warp, 8 warps, pieces), 256 experts, 8 more
    tol = 2 * z_tol(logits) + (13 + T / 8 + 8 + T / 32 + 4 + 13 + 8) * U
    assert (np.abs(f64(loss) - lr) <= tol * lr).all()
    dloss = torch.randn(n_seq, generator=torch.Generator().manual_seed(1))
    (dl, cd) = guarded_empty((T, Nr), torch.float32)
    for d in (dloss, None):
        bal = dict(seq_offsets=offd, counts=counts, dloss=None if d is None else d.cuda(), alpha=0.3)
        m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), balance=bal, dlogits=dl, err=err)
        cd()
        ref, mag = O.router_dlogits(z, idx.numpy().astype(np.int64), off=off, counts=cr,
                                    dloss=None if d is None else d.numpy(), alpha=0.3)
        # p: sum s of 13 and a product; sum f p: 13 more; 8 products around them
        assert (np.abs(f64(dl) - ref) <= (4 * z_tol(logits) + (13 + 1 + 13 + 8) * U) * mag + 2.0 ** -140).all()
    assert m.moe_check_device_error(err)[0] == m.MOE_OK


@pytest.mark.parametrize("T,Nr,Kr,S,off", CASES)
@pytest.mark.parametrize("H", [128, 640])
def test_router_backward(m, T, Nr, Kr, S, off, H):
    logits, idx = router_inputs(T, Nr, Kr, S, T + 1)
    rs = 2.5
    cfg = m.config(H, 128, Nr, Kr, route_scale=rs)
    g = torch.Generator().manual_seed(H)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    wr = (torch.randn((Nr, H), generator=g) * 0.02).to(torch.bfloat16)
    dgate = torch.randn((T, Kr), generator=g)
    idn = idx.numpy().astype(np.int64)
    counts = O.seq_counts(idn, off, Nr)
    bal = dict(seq_offsets=torch.tensor(off, dtype=torch.int32).cuda(),
               counts=torch.tensor(counts, dtype=torch.int32).cuda(), alpha=0.3)
    (dl, c1), (dx, c2), (dwr, c3) = (guarded_empty((T, Nr), torch.float32), guarded_empty((T, H), torch.float32),
                                     guarded_empty((Nr, H), torch.float32))
    err = m.new_err_flag()
    args = dict(x=x.cuda(), wr=wr.cuda(), dgate=dgate.cuda(), balance=bal, err=err)
    m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dlogits=dl, dx=dx, dwr=dwr, **args)
    c1(), c2(), c3()
    assert m.moe_check_device_error(err)[0] == m.MOE_OK
    ref, mag = O.router_dlogits(logits.double().sum(0).numpy(), idn, dgate=dgate.numpy(), route_scale=rs, off=off,
                                counts=counts, alpha=0.3)
    dz_tol = (4 * z_tol(logits) + (13 + 1 + 13 + 8) * U) * mag
    assert (np.abs(f64(dl) - ref) <= dz_tol + 2.0 ** -140).all()
    # the products of the GPU's own dz: three parts of 16-long tensor-core steps into one FP32 accumulator (each step
    # off by at most two FP32 steps of the running sum's magnitude), the token ranges' join
    dz = f64(dl)
    Np, nt = (Nr + 63) // 64 * 64, (T + 31) // 32 * 32
    wx, xx = f64(wr), f64(x)
    assert (np.abs(f64(dx) - dz @ wx) <= (3 * Np / 16 + 2) * 4 * U * (np.abs(dz) @ np.abs(wx))).all()
    assert (np.abs(f64(dwr) - dz.T @ xx) <= (3 * nt / 16 + 150) * 4 * U * (np.abs(dz).T @ np.abs(xx))).all()
    # again, added to what is there, and each output by itself: the same bits
    base = torch.randn((T, H), generator=g).cuda()
    acc = base.clone()
    _, a, _ = m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dx=acc, dx_accumulate=True, **args)
    assert torch.equal(a, base + dx)
    assert torch.equal(m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dwr=True, **args)[2], dwr)


def test_router_products_keep_24_bits(m):
    """One token: dW_r = dz x has a single term, so losing any part of dz would show."""
    logits, idx = router_inputs(1, 256, 8, 1, 9)
    cfg = m.config(512, 128, 256, 8)
    x = torch.randn((1, 512), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    dgate = torch.randn((1, 8), generator=torch.Generator().manual_seed(3)).cuda()
    dl, _, dwr = m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), x=x, dgate=dgate, dlogits=True, dwr=True)
    ref = f64(dl).T @ f64(x)
    assert (np.abs(f64(dwr) - ref) <= 8 * U * np.abs(ref)).all()


def test_far_logits(m):
    """Affinities that underflow, and ones next to 1: finite gradients, 1 - s with its digits."""
    Nr, Kr = 16, 4
    z = torch.full((3, Nr), -200.0)   # every affinity 0
    z[1] = 30.0                       # 1 - s = 9e-14
    z[2, :8], z[2, 8:] = 30.0, -200.0
    idx = torch.arange(Kr, dtype=torch.int32).repeat(3, 1)
    cfg = m.config(128, 128, Nr, Kr)
    dgate = torch.randn((3, Kr), generator=torch.Generator().manual_seed(0))
    off = torch.tensor([0, 3], dtype=torch.int32).cuda()
    loss, counts = m.moe_balance_loss(cfg, z[None].cuda(), idx.cuda(), off)
    assert torch.isfinite(loss).all()
    dl, _, _ = m.moe_router_backward(cfg, z[None].cuda(), idx.cuda(), dgate=dgate.cuda(), dlogits=True,
                                     balance=dict(seq_offsets=off, counts=counts, alpha=0.3))
    assert torch.isfinite(dl).all() and (dl[0] == 0).all()
    ref, mag = O.router_dlogits(z[1:].double().numpy(), idx[1:].numpy().astype(np.int64), dgate=dgate[1:].numpy())
    g, _, _ = m.moe_router_backward(cfg, z[None].cuda(), idx.cuda(), dgate=dgate.cuda(), dlogits=True)
    assert (np.abs(f64(g)[1:] - ref) <= (4 * (200 + 7) + 40) * U * mag + 1e-40).all()


def test_router_bad_indices_and_repeats(m):
    logits, idx = router_inputs(6, 16, 4, 1, 4)
    cfg = m.config(128, 128, 16, 4)
    off = torch.tensor([0, 6], dtype=torch.int32).cuda()
    dgate = torch.randn((6, 4), generator=torch.Generator().manual_seed(0))
    # the same expert twice in a token: both slots' gradients land on it
    idx[2, 1] = idx[2, 0]
    err = m.new_err_flag()
    dl, _, _ = m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dgate=dgate.cuda(), dlogits=True, err=err)
    ref, mag = O.router_dlogits(logits.double().sum(0).numpy(), idx.numpy().astype(np.int64), dgate=dgate.numpy())
    assert (np.abs(f64(dl) - ref) <= (4 * z_tol(logits) + 40 * U) * mag + 1e-40).all()
    assert m.moe_check_device_error(err)[0] == m.MOE_OK
    idx[4, 2] = -1
    idx[5, 0] = 16
    _, counts = m.moe_balance_loss(cfg, logits.cuda(), idx.cuda(), off, err=err)
    assert m.moe_check_device_error(err) == (m.MOE_ERR_DEVICE, m.MOE_DEVERR_BAD_INDEX)
    assert np.array_equal(counts.cpu().numpy(), O.seq_counts(idx.numpy(), [0, 6], 16))
    err = m.new_err_flag()
    dl, _, _ = m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dgate=dgate.cuda(), dlogits=True, err=err)
    assert m.moe_check_device_error(err) == (m.MOE_ERR_DEVICE, m.MOE_DEVERR_BAD_INDEX)
    assert torch.isfinite(dl).all()


@pytest.mark.parametrize("off", [[0, 9, 4, 10], [0, 400], [-3, 5], [5, 3]])
def test_wrong_offsets_are_reported(m, off):
    logits, idx = router_inputs(10, 16, 4, 1, 4)
    cfg = m.config(128, 128, 16, 4)
    err = m.new_err_flag()
    offd = torch.tensor(off, dtype=torch.int32).cuda()
    m.moe_balance_loss(cfg, logits.cuda(), idx.cuda(), offd, err=err)
    assert m.moe_check_device_error(err) == (m.MOE_ERR_DEVICE, m.MOE_DEVERR_BAD_INDEX)


def test_empty_batches(m):
    cfg = m.config(128, 128, 16, 4)
    logits, idx = torch.empty((1, 0, 16), device="cuda"), torch.empty((0, 4), dtype=torch.int32, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    loss, counts = m.moe_balance_loss(cfg, logits, idx, off)
    assert (loss == 0).all() and (counts == 0).all()
    dwr = torch.full((16, 128), 3.0, device="cuda")
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    wr = torch.zeros((16, 128), dtype=torch.bfloat16, device="cuda")
    dl, dx, dwr = m.moe_router_backward(cfg, logits, idx, x=x, wr=wr, dlogits=True, dx=True, dwr=dwr)
    assert (dwr == 0).all() and dl.shape == (0, 16) and dx.shape == (0, 128)


def test_route_then_backward(m):
    """moe_route's own state feeds the loss and the backward: the gates it gave are those the gradient is of."""
    import moe_synth as S
    T, H, Nr, Kr = 200, 512, 16, 4
    cfg = m.config(H, 128, Nr, Kr, route_scale=1.5)
    x, wr, bias = S.gen_x(T, H, 1).cuda(), S.gen_router(Nr, H, 1).cuda(), S.gen_bias(Nr, 1).cuda()
    ws = torch.empty(m.moe_route_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    idx, gate, _ = m.moe_route(cfg, x, wr, bias, ws=ws)
    logits = m.moe_route_logits(cfg, T, ws)
    z = logits.double().sum(0)
    s = torch.sigmoid(z).gather(1, idx.long())
    assert torch.allclose(1.5 * s / s.sum(1, keepdim=True), gate.double(), rtol=1e-5, atol=0)
    dgate = torch.randn((T, Kr), generator=torch.Generator().manual_seed(0)).cuda()
    dl, dx, dwr = m.moe_router_backward(cfg, logits, idx, x=x, wr=wr, dgate=dgate, dlogits=True, dx=True, dwr=True)
    ref, mag = O.router_dlogits(z.cpu().numpy(), idx.cpu().numpy().astype(np.int64), dgate=dgate.cpu().numpy(),
                                route_scale=1.5)
    assert (np.abs(f64(dl) - ref) <= (4 * z_tol(logits.cpu()) + 40 * U) * mag + 1e-40).all()


def test_captured_replays_on_another_stream(m):
    """One capture of the whole chain, replayed on new inputs in the same buffers."""
    T, H, Nr, Kr = 150, 512, 16, 4
    cfg = m.config(H, 128, Nr, Kr)
    off = torch.tensor([0, 60, 150], dtype=torch.int32).cuda()
    xs = [torch.randn((T, H), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(2)]
    wr = (torch.randn((Nr, H), generator=torch.Generator().manual_seed(7)) * 0.02).to(torch.bfloat16).cuda()
    logits, idx = (t.cuda() for t in router_inputs(T, Nr, Kr, 2, 5))
    dgate = torch.randn((T, Kr), generator=torch.Generator().manual_seed(8)).cuda()
    x, err = xs[0].clone(), m.new_err_flag()

    def chain():
        h, y, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, x, None, EPS)
        loss, counts = m.moe_balance_loss(cfg, logits, idx, off, err=err)
        _, dx, dwr = m.moe_router_backward(cfg, logits, idx, x=y, wr=wr, dgate=dgate, dx=True, dwr=True, err=err,
                                           balance=dict(seq_offsets=off, counts=counts))
        dh, dw = m.add_rmsnorm_backward(dx, h, rstd)
        return q, s, loss, dwr, dh, dw

    want = []
    for v in xs:
        x.copy_(v)
        want.append([t.clone() for t in chain()])
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        got = chain()
    for v, w in zip(xs, want):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    assert m.moe_check_device_error(err)[0] == m.MOE_OK


def test_many_short_sequences(m):
    """More sequences than a grid's second dimension holds, most of them empty or one token long."""
    T, Nr, Kr = 400, 16, 4
    logits, idx = router_inputs(T, Nr, Kr, 1, 6)
    cfg = m.config(128, 128, Nr, Kr)
    off = torch.sort(torch.randint(0, T + 1, (70001,), generator=torch.Generator().manual_seed(0))).values
    err = m.new_err_flag()
    offd = off.to(torch.int32).cuda()
    loss, counts = m.moe_balance_loss(cfg, logits.cuda(), idx.cuda(), offd, alpha=0.3, err=err)
    z = logits.double().sum(0).numpy()
    o = off.numpy()
    lr, cr = O.balance_loss(z, idx.numpy().astype(np.int64), o, 0.3)
    assert np.array_equal(counts.cpu().numpy(), cr)
    assert (np.abs(f64(loss) - lr) <= (2 * z_tol(logits) + 60 * U) * lr).all()
    dl, _, _ = m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dlogits=True, err=err,
                                     balance=dict(seq_offsets=offd, counts=counts, alpha=0.3))
    ref, mag = O.router_dlogits(z, idx.numpy().astype(np.int64), off=o, counts=cr, alpha=0.3)
    assert (np.abs(f64(dl) - ref) <= (4 * z_tol(logits) + 40 * U) * mag + 1e-40).all()
    assert m.moe_check_device_error(err)[0] == m.MOE_OK


def test_on_a_stream_of_ones_own(m):
    """A stream given by object or by handle: workspaces and outputs belong to it, results are the same."""
    T, H, Nr, Kr = 300, 512, 16, 4
    cfg = m.config(H, 128, Nr, Kr)
    logits, idx = (t.cuda() for t in router_inputs(T, Nr, Kr, 2, 5))
    g = torch.Generator().manual_seed(0)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn((Nr, H), generator=g) * 0.02).to(torch.bfloat16).cuda()
    dgate = torch.randn((T, Kr), generator=g).cuda()
    off = torch.tensor([0, 100, 300], dtype=torch.int32).cuda()

    def chain(**kw):
        h, y, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, x, None, EPS, **kw)
        loss, counts = m.moe_balance_loss(cfg, logits, idx, off, **kw)
        _, dx, dwr = m.moe_router_backward(cfg, logits, idx, x=y, wr=wr, dgate=dgate, dx=True, dwr=True,
                                           balance=dict(seq_offsets=off, counts=counts), **kw)
        return [q, s, loss, dwr, *m.add_rmsnorm_backward(dx, h, rstd, **kw)]

    want = chain()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (st, st.cuda_stream, 0):
        for _ in range(3):
            got = chain(stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(m):
    """Two calls of each kind under way at the same time keep their results."""
    T, H, Nr, Kr = 2000, 1024, 64, 4
    cfg = m.config(H, 128, Nr, Kr)
    sets = []
    for k in range(2):
        g = torch.Generator().manual_seed(k)
        logits, idx = (t.cuda() for t in router_inputs(T, Nr, Kr, 1, k))
        sets.append((logits, idx, torch.randn((T, H), generator=g).to(torch.bfloat16).cuda(),
                     (torch.randn((Nr, H), generator=g) * 0.02).to(torch.bfloat16).cuda(),
                     torch.randn((T, Kr), generator=g).cuda()))

    def chain(logits, idx, x, wr, dgate):
        h, y, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, x, None, EPS)
        _, dx, dwr = m.moe_router_backward(cfg, logits, idx, x=y, wr=wr, dgate=dgate, dx=True, dwr=True)
        return [q, s, dwr, *m.add_rmsnorm_backward(dx, h, rstd)]

    want = [chain(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = chain(*sets[k])
    torch.cuda.synchronize()
    for g_, w_ in zip(got, want):
        for a, b in zip(g_, w_):
            assert torch.equal(a, b)


def test_router_outputs_at_their_least_alignment(m):
    """dx and dwr 16 bytes into a sector, dlogits and its inputs on odd words: the same bits as aligned ones."""
    T, H, Nr, Kr = 300, 384, 100, 5
    cfg = m.config(H, 128, Nr, Kr)
    logits, idx = (t.cuda() for t in router_inputs(T, Nr, Kr, 2, 8))
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn((Nr, H), generator=g) * 0.02).to(torch.bfloat16).cuda()
    dgate = torch.randn((T, Kr), generator=g).cuda()

    def off(n, shape, src=None, dtype=torch.float32):
        size = int(np.prod(shape))
        t = torch.empty(size + n, dtype=dtype, device="cuda")[n:].view(shape)
        return t if src is None else t.copy_(src)

    want = m.moe_router_backward(cfg, logits, idx, x=x, wr=wr, dgate=dgate, dlogits=True, dx=True, dwr=True)
    dx, dwr, dl = off(4, (T, H)), off(4, (Nr, H)), off(1, (T, Nr))
    assert dx.data_ptr() % 32 == 16 and dl.data_ptr() % 16 == 4
    got = m.moe_router_backward(cfg, off(4, logits.shape, logits), off(1, idx.shape, idx, torch.int32),
                                x=off(8, x.shape, x, torch.bfloat16), wr=off(8, wr.shape, wr, torch.bfloat16),
                                dgate=off(1, dgate.shape, dgate), dlogits=dl, dx=dx, dwr=dwr)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # logits off a 16-byte boundary are refused
    with pytest.raises(m.MoeError):
        m.moe_router_backward(cfg, off(1, logits.shape, logits), idx, dgate=dgate, dlogits=True)


def test_bindings_refuse_wrong_tensors(m):
    T, H, Nr, Kr = 4, 256, 16, 4
    cfg = m.config(H, 128, Nr, Kr)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    f = torch.zeros((T, H), device="cuda")
    r = torch.ones(T, device="cuda")
    z, idx = torch.zeros((1, T, Nr), device="cuda"), torch.zeros((T, Kr), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    wr = torch.zeros((Nr, H), dtype=torch.bfloat16, device="cuda")
    n, b, l, w = m.fp8_add_rmsnorm_quant_1x128, m.add_rmsnorm_backward, m.moe_balance_loss, m.moe_router_backward
    counts = torch.zeros((1, Nr), dtype=torch.int32, device="cuda")
    bad = [
        lambda: n(x.half()), lambda: n(x.t()), lambda: n(x[0]), lambda: n(x, f), lambda: n(x, x[:2]),
        lambda: n(x, x.cpu()), lambda: n(x, None, torch.ones(H, device="cuda", dtype=torch.bfloat16)),
        lambda: n(x, None, torch.ones(H)), lambda: n(x, y=f), lambda: n(x, q=torch.zeros((T, H), device="cuda")),
        lambda: n(x, scales=torch.zeros((T, 3), device="cuda")), lambda: n(x, rstd=torch.zeros(T + 1, device="cuda")),
        lambda: n(x, x, h=f), lambda: n(x[:, :250]), lambda: n(None), lambda: n(x, eps=0.0), lambda: n(x[:, 1:129]),
        lambda: b(f, x, r[:2]), lambda: b(f.half(), x, r), lambda: b(f, x, r, dres=f), lambda: b(f, x, r, dx=f.half()),
        lambda: b(f, x, r, dx=f, dx_dtype=torch.bfloat16), lambda: b(f, x.t(), r), lambda: b(f[:2], x, r),
        lambda: b(f, x, r, ws=torch.zeros(8, dtype=torch.uint8, device="cuda")), lambda: b(f, x, r, dx_dtype=torch.half),
        lambda: b(f, x, r, dw=torch.zeros(H + 1, device="cuda")), lambda: b(f, x, r, dx_dtype="bf16"),
        lambda: l(cfg, z[0], idx, off), lambda: l(cfg, z, idx.long(), off), lambda: l(cfg, z, idx, off.long()),
        lambda: l(cfg, z, idx[:2], off), lambda: l(cfg, z, idx, off[:0]), lambda: l(cfg, z[:, :, :8], idx, off),
        lambda: l(cfg, z, idx, off, loss=r), lambda: l(cfg, z, idx, off, alpha=float("nan")),
        lambda: l(cfg, z, idx, off, counts=torch.zeros((1, Nr), device="cuda")),
        lambda: w(cfg, z, idx, dwr=True), lambda: w(cfg, z, idx, dx=True), lambda: w(cfg, z, idx, x=f, dwr=True),
        lambda: w(cfg, z, idx, dgate=f, dlogits=True), lambda: w(cfg, z, idx, wr=wr, dx=True, dx_accumulate=True),
        lambda: w(cfg, z, idx, dlogits=f), lambda: w(cfg, z, idx, balance=dict(seq_offsets=off), dlogits=True),
        lambda: w(cfg, z, idx, balance=dict(seq_offsets=off, counts=counts[:, :8]), dlogits=True),
        lambda: w(cfg, z, idx, balance=dict(seq_offsets=off, counts=counts, dloss=f), dlogits=True),
        lambda: w(cfg, z, idx, balance=[off, counts], dlogits=True),
        lambda: w(cfg, z, idx, wr=wr, dx=True, ws=torch.zeros(8, dtype=torch.uint8, device="cuda")),
    ]
    for i, f_ in enumerate(bad):
        with pytest.raises(m.MoeError):
            f_()
            pytest.fail(f"case {i} was not refused")
    # and what is asked for in its least form works
    assert w(cfg, z, idx) == (None, None, None)
    assert w(cfg, z, idx, wr=wr, dx=True)[1].abs().sum() == 0
    torch.cuda.synchronize()

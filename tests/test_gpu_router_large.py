"""The operators around the layer where their kernels' loops turn over: several
units a pair of CTAs, several accumulations a run, several tokens a warp, and
workspaces of exactly the reported size.

The products are compared with 64-bit products of the call's own dz by their
relative norm.  A tensor-core step drops less than 2^-23 of the accumulator,
whose root-mean-square size after k of n steps is sqrt(k / n) of the result's:
2/3 n 2^-23 over n steps.  Losing dz's third part (16 bits are left, cut off
towards zero) would show as about 8e-6, an accumulator kept over a whole run of
tokens as 5e-6 and more.
"""
import numpy as np
import pytest
import torch

from _moe_util import guarded_empty
from oracle import block as O
from test_gpu_block import EPS, problem
from test_gpu_operators import U, f64, router_inputs, z_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def steps_tol(n):
    return 2 / 3 * n * 2.0 ** -23


def cuts(T, n, g, first=0, last=None):
    """n sequences with borders anywhere, some of them empty."""
    off = torch.randint(first, (last or T) + 1, (n + 1,), generator=g).sort().values
    off[1 + n // 3] = off[n // 3]
    off[0], off[-1] = first, last or T
    return off.sort().values


@pytest.mark.parametrize("T,H,Nr,Kr", [(6001, 7168, 256, 8),   # side by side, 18 units a pair, 24 token tiles
                                       (12001, 7168, 256, 8),  # one after the other
                                       (6001, 7168, 64, 4),    # the same with few experts
                                       (9000, 640, 100, 5)])   # odd strips, experts behind N_r
def test_products_of_long_batches(m, T, H, Nr, Kr):
    g = torch.Generator().manual_seed(T + Nr)
    logits, idx = (t.cuda() for t in router_inputs(T, Nr, Kr, 1, T))
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn((Nr, H), generator=g) * 0.02).to(torch.bfloat16).cuda()
    dgate = torch.randn((T, Kr), generator=g).cuda()
    cfg = m.config(H, 128, Nr, Kr)
    err = m.new_err_flag()
    nbytes = m.lib.moe_router_backward_workspace_size(m._binding.C.byref(cfg), T)
    ws, cws = guarded_empty((nbytes,), torch.uint8)
    (dl, c1), (dx, c2), (dwr, c3) = (guarded_empty((T, Nr), torch.float32), guarded_empty((T, H), torch.float32),
                                     guarded_empty((Nr, H), torch.float32))
    kw = dict(x=x, wr=wr, dgate=dgate, err=err)
    m.moe_router_backward(cfg, logits, idx, dlogits=dl, dx=dx, dwr=dwr, ws=ws, **kw)
    cws(), c1(), c2(), c3()
    dz = dl.double()
    want = dz @ wr.double()
    # three products a step of 16 experts, every 64-expert block of the parts; one rounding more for what is stored
    n = 3 * ((Nr + 63) // 64 * 64) // 16
    assert (dx.double() - want).norm() <= (steps_tol(n) + U) * want.norm()
    tile = (dx.double() - want).view(T, H // 128, 128).norm(dim=2)
    # no 128-column piece of a row is off on its own (its size varies less than 8-fold from the mean's)
    assert tile.max() <= 8 * 4 * (steps_tol(n) + U) * want.norm() / (T * H / 128) ** 0.5
    wantw = dz.t() @ x.double()
    # 24 steps an accumulation; then one FP32 addition each per accumulation of a run and per piece of the join
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    strips, stages = (H + 255) // 256, (T + 63) // 64
    run = -(-strips * stages // pairs)
    adds = (run + 1) // 2 + 1 + stages // max(run, 1) + 2
    assert (dwr.double() - wantw).norm() <= (steps_tol(24) + 2 / 3 * adds * U) * wantw.norm()
    # each product by itself, and dx added to what is there: the same bits
    assert torch.equal(m.moe_router_backward(cfg, logits, idx, dwr=True, **kw)[2], dwr)
    assert torch.equal(m.moe_router_backward(cfg, logits, idx, dx=True, **kw)[1], dx)
    base = torch.randn((T, H), generator=g).cuda()
    acc = base.clone()
    _, _, w2 = m.moe_router_backward(cfg, logits, idx, dx=acc, dx_accumulate=True, dwr=True, **kw)
    assert torch.equal(acc, base + dx) and torch.equal(w2, dwr)
    assert m.moe_check_device_error(err)[0] == m.MOE_OK


def test_dx_keeps_24_bits(m):
    """One expert's row of W_r alone: dx = dz_e w_e has a single term."""
    T, H, Nr, Kr = 700, 512, 256, 8
    logits, idx = (t.cuda() for t in router_inputs(T, Nr, Kr, 1, 9))
    cfg = m.config(H, 128, Nr, Kr)
    g = torch.Generator().manual_seed(2)
    dgate = torch.randn((T, Kr), generator=g).cuda()
    bal = dict(seq_offsets=torch.tensor([0, 300, T], dtype=torch.int32).cuda(), alpha=3.0)
    bal["counts"] = m.moe_balance_loss(cfg, logits, idx, bal["seq_offsets"])[1]
    for e in (0, 37, 255):
        wr = torch.zeros((Nr, H), dtype=torch.bfloat16, device="cuda")
        wr[e] = torch.randn((H,), generator=g).to(torch.bfloat16)
        dl, dx, _ = m.moe_router_backward(cfg, logits, idx, wr=wr, dgate=dgate, balance=bal, dlogits=True, dx=True)
        ref = dl[:, e].double()[:, None] * wr[e].double()
        assert ((dx.double() - ref).abs() <= 8 * U * ref.abs()).all()


@pytest.mark.parametrize("T,Nr,Kr,S,n_seq", [(40009, 256, 8, 1, 2000), (40009, 33, 4, 5, 17), (6000, 256, 8, 2, 900),
                                             (20001, 128, 6, 4, 1)])
def test_balance_of_long_batches(m, T, Nr, Kr, S, n_seq):
    """Several tokens a warp, with sequence borders inside its run, and tokens outside every sequence."""
    g = torch.Generator().manual_seed(T + Nr)
    logits, idx = router_inputs(T, Nr, Kr, S, T + Nr)
    off = cuts(T, n_seq, g, first=3, last=T - 5)
    offd = off.to(torch.int32).cuda()
    cfg = m.config(128, 128, Nr, Kr)
    err = m.new_err_flag()
    nbytes = m.lib.moe_balance_loss_workspace_size(m._binding.C.byref(cfg), T, n_seq)
    ws, cws = guarded_empty((nbytes,), torch.uint8)
    (loss, cl), (counts, cc) = guarded_empty((n_seq,), torch.float32), guarded_empty((n_seq, Nr), torch.int32)
    m.moe_balance_loss(cfg, logits.cuda(), idx.cuda(), offd, alpha=0.3, loss=loss, counts=counts, ws=ws, err=err)
    cws(), cl(), cc()
    z, idn, o = logits.double().sum(0).numpy(), idx.numpy().astype(np.int64), off.numpy()
    lr, cr = O.balance_loss(z, idn, o, 0.3)
    assert np.array_equal(counts.cpu().numpy(), cr)
    # sum s: 8 + 5; a warp's tokens of a chunk (T / 592 / 8 + 1), 8 warps, every 64th piece, 6 more; experts 13, CTAs 8
    chain = 13 + T / 592 / 8 + 2 + 8 + (T / 8 / 64 + 1) + 6 + 13 + 8 + 8
    assert (np.abs(f64(loss) - lr) <= (2 * z_tol(logits) + chain * U) * lr).all()
    dloss = torch.randn(n_seq, generator=g)
    dgate = torch.randn((T, Kr), generator=g)
    dl, cd = guarded_empty((T, Nr), torch.float32)
    m.moe_router_backward(cfg, logits.cuda(), idx.cuda(), dgate=dgate.cuda(), dlogits=dl, err=err,
                          balance=dict(seq_offsets=offd, counts=counts, dloss=dloss.cuda(), alpha=0.3))
    cd()
    ref, mag = O.router_dlogits(z, idn, dgate=dgate.numpy(), off=o, counts=cr, dloss=dloss.numpy(), alpha=0.3)
    assert (np.abs(f64(dl) - ref) <= (4 * z_tol(logits) + 40 * U) * mag + 1e-40).all()
    assert m.moe_check_device_error(err)[0] == m.MOE_OK


@pytest.mark.parametrize("T,H", [(5, 128), (700, 1024), (3000, 7168), (9, 16384)])
def test_norm_backward_workspace(m, T, H):
    g = torch.Generator().manual_seed(T)
    h, dy = (torch.randn((T, H), generator=g).cuda() for _ in range(2))
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    nbytes = m.lib.add_rmsnorm_backward_workspace_size(T, H)
    ws, check = guarded_empty((nbytes,), torch.uint8)
    dx, dw = m.add_rmsnorm_backward(dy, h, rstd, ws=ws)
    check()
    n = h.double() * rstd.double()[:, None]
    want = (dy.double() * n).sum(0)
    # at most T rows in a chain, 8 row groups, the CTAs in 32 chains, 32 more; 2 products
    assert ((dw.double() - want).abs() <= (T + 8 + 40 + 32 + 2) * U * (dy.double() * n).abs().sum(0)).all()


@pytest.mark.parametrize("T", [1, 300])
def test_block_workspaces(m, T):
    """Guard bands around the block's workspaces (build_gpu_layer asks for them)."""
    cfg, layer, x, resid, w, dout = problem(m, T, 41)
    assert layer.guard_bytes
    off = torch.tensor([0, T // 2, T], dtype=torch.int32).cuda()
    _, saved = layer.block_forward(x, resid, w, EPS)
    _, bal = layer.balance_loss(T, off)
    layer.block_backward(saved, dout, balance=bal)
    layer.backward(saved["y"], dout)
    assert len(layer._guarded) == 3
    layer.check_guards()
    layer.check()


def deq(codes, scales):
    """E4M3 codes with a scale per 128 columns (and per 128 rows, where scales has fewer rows), in 64 bits."""
    v = codes.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, -1)
    return v * (s if s.shape[0] == v.shape[0] else s.repeat_interleave(128, 0))


def test_gate_gradient_from_the_codes(m):
    """The whole chain from the codes of y, dout and the weights to dW_r: G, U, dh, g dL/dg, dz in 64 bits."""
    T = 96
    cfg, layer, x, resid, w, dout = problem(m, T, 43)
    H, I, Nr, Kr = cfg["H"], cfg["I"], cfg["Nr"], cfg["Kr"]
    _, saved = layer.block_forward(x, resid, w, EPS)
    got = layer.block_backward(saved, dout)["dwr"].double()
    ws, L = layer.workspace(T), layer.layout(T)
    X = deq(m.ws_view(ws, L, "xq", torch.uint8, (T, H)), m.ws_view(ws, L, "xs", torch.float32, (T, H // 128)))
    D = deq(*m.fp8_quant_1x128(dout))
    gate = m.ws_view(ws, L, "gate", torch.float32, (T, Kr)).double()
    logits, idx = layer.router_state(T)
    # an FP8 product over K: 4 truncating steps a 128-long partial (two FP32 steps each), its scale and promotion
    gemm = lambda K: (4 * 4 + 4 + K / 128) * U  # noqa: E731
    a, a_err, a_mag = (torch.zeros((T, Kr), dtype=torch.float64, device="cuda") for _ in range(3))
    for e in range(Nr):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        W13, W2 = deq(layer.w13[e], layer.s13[e]), deq(layer.w2[e], layer.s2[e])
        GU, GUe = X[t] @ W13.t(), gemm(H) * (X[t].abs() @ W13.abs().t())
        G, Up, Ge, Ue = GU[:, :I], GU[:, I:], GUe[:, :I], GUe[:, I:]
        silu = G * torch.sigmoid(G)
        h, he = silu * Up, 1.1 * Up.abs() * Ge + silu.abs() * Ue  # |silu'| < 1.1
        g = gate[t, k][:, None]
        dh, dhe = g * (D[t] @ W2), g * gemm(H) * (D[t].abs() @ W2.abs())
        a[t, k] = (dh * h).sum(1)
        a_mag[t, k] = (dh * h).abs().sum(1)
        a_err[t, k] = (dh.abs() * he + h.abs() * dhe).sum(1)
    a_err = a_err + (8 + 9 + I / 128) * U * a_mag
    z, idn = f64(logits).sum(0), idx.cpu().numpy().astype(np.int64)
    dz, mag = O.router_dlogits(z, idn, dgate=f64(a / gate))
    _, dze = O.router_dlogits(z, idn, dgate=f64(a_err / gate))  # the magnitudes: om (err + gh sum err)
    dze = torch.from_numpy(dze + (4 * z_tol(logits.cpu()) + 40 * U) * mag).cuda()
    dz, y = torch.from_numpy(dz).cuda(), saved["y"].double()
    bound = dze.t() @ y.abs() + (3 * 96 / 16 + 20) * 4 * U * (dz.abs().t() @ y.abs())
    assert ((got - dz.t() @ y).abs() <= bound).all()
    # that bound adds every rounding up one way (2^-7 of the result); by size, G, U and dh are off by their steps and
    # additions (G's error counts twice through silu), a by its own sum, dz and the product as above
    gemm_rms = 2 / 3 * 4 * 2.0 ** -23 + (H / 128 + 3) * U
    rel = 4 * gemm_rms + (8 + 9 + I / 128) * U + 4 * z_tol(logits.cpu()) + 40 * U + steps_tol(24) + 8 * U
    assert (got - dz.t() @ y).norm() <= rel * got.norm() and rel < 2.0 ** -15

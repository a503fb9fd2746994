"""The block (norm in front of the layer, and its whole backward): the
operators together, as a training step runs them.  Each stage is compared with
the operator that computes it alone or, from the call's own FP32 intermediates,
with the 64-bit oracle; tolerances count roundings as in
test_gpu_operators.py."""
import numpy as np
import pytest
import torch

import moe_synth as S
from _moe_util import Problem
from oracle import block as O
from test_gpu_layer import build_gpu_layer
from test_gpu_operators import EPS, U, f64, half, z_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def problem(m, T, seed, **over):
    cfg = dict(S.TINY, **over)
    prob = Problem(cfg, T, seed=seed)
    layer = build_gpu_layer(m, prob)
    H = cfg["H"]
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, H), generator=g) * 0.5).to(torch.bfloat16).cuda()
    resid = (torch.randn((T, H), generator=g) * 2).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn((H,), generator=g)).cuda()
    dout = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    return cfg, layer, x, resid, w, dout


@pytest.mark.parametrize("T,over", [(1, {}), (129, {}), (300, dict(n_groups=4, topk_groups=2)), (64, dict(Ns=0)),
                                    (40, dict(scale_mode=1))])
def test_block_forward(m, T, over):
    cfg, layer, x, resid, w, _ = problem(m, T, 3, **over)
    pow2 = layer.cfg.scale_mode == m.MOE_SCALE_POW2
    idx = torch.empty((T, cfg["Kr"]), dtype=torch.int32, device="cuda")
    counts = torch.empty((cfg["Nr"],), dtype=torch.int32, device="cuda")
    out, saved = layer.block_forward(x, resid, w, EPS, out_dtype=m.MOE_DTYPE_F32, idx_out=idx, counts_out=counts)
    layer.check()
    # the norm and its codes, bit for bit, in the workspace's places
    h, y, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, resid, w, EPS, pow2=pow2)
    ws, L = layer.workspace(T), layer.layout(T)
    xq = m.ws_view(ws, L, "xq", torch.uint8, q.shape)
    xs = m.ws_view(ws, L, "xs", torch.float32, s.shape)
    for a, b in ((saved["h"], h), (saved["y"], y), (saved["rstd"], rstd), (xq, q), (xs, s)):
        assert torch.equal(a, b)
    # the routing is that of y
    ridx, gate, rcounts = m.moe_route(layer.cfg, y, layer.wr, layer.bias)
    assert torch.equal(ridx, idx) and torch.equal(rcounts, counts)
    assert torch.equal(m.ws_view(ws, L, "gate", torch.float32, gate.shape), gate)
    # the experts on those codes through the packed rows of expert parallelism, on the residual h
    cfgl, H, Kr = layer.cfg, cfg["H"], cfg["Kr"]
    nb = m.moe_ep_row_bytes(cfgl)
    send = torch.empty((T, nb), dtype=torch.uint8, device="cuda")
    selfr = torch.empty((T, nb), dtype=torch.uint8, device="cuda")
    cnt, off = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    row_of = torch.empty((T, 1), dtype=torch.int32, device="cuda")
    m.moe_ep_dispatch(cfgl, 1, q, s, idx, gate, send, cnt, off, row_of, self_rows=selfr, err=layer.err)
    W, Nr = layer.weights(), cfg["Nr"]
    part = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    loc = m.config(H, cfg["I"], Nr, Kr, 0, scale_mode=cfgl.scale_mode)
    m.moe_ep_experts(loc, {k: (W[k] if k == "wr" else W[k][:Nr]) for k in W}, send, part, err=layer.err)
    ref = h.double() + part.double()[row_of[:, 0].long()]
    # each partial sum is a bf16 rounding of an FP32 sum of at most 16 terms
    tol = half(torch.bfloat16) * part.double().abs()[row_of[:, 0].long()]
    if cfg.get("Ns", 1):
        sh = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        loc1 = m.config(H, cfg["I"], 1, Kr, 0, scale_mode=cfgl.scale_mode)
        m.moe_ep_experts(loc1, {k: (W[k] if k == "wr" else W[k][Nr:]) for k in W}, selfr, sh, err=layer.err)
        ref = ref + sh.double()
        tol = tol + half(torch.bfloat16) * sh.double().abs()
    layer.check()
    y_rows = m.ws_view(ws, L, "y", torch.float32, (T * (Kr + cfg.get("Ns", 1)), H))
    pos = m.ws_view(ws, L, "pos", torch.int32, (T, Kr)).long()
    mag = h.double().abs() + y_rows[pos].double().abs().sum(1)
    if cfg.get("Ns", 1):
        mag = mag + y_rows[T * Kr:].double().abs()
    assert ((out.double() - ref).abs() <= tol * 1.01 + 40 * U * mag).all()
    # without a residual stream: h is x
    out1, saved1 = layer.block_forward(x, None, w, EPS)
    assert saved1["h"] is x and out1.dtype == torch.bfloat16


@pytest.mark.parametrize("T,over,off", [(300, {}, [0, 100, 100, 290]), (1, {}, None), (129, dict(route_scale=2.5), [0, 129]),
                                        (70, dict(Ns=0), None), (200, dict(n_groups=4, topk_groups=2), [0, 64, 200]),
                                        (600, dict(H=1152, I=384, Nr=72, Kr=8), [0, 5, 400, 600])])
def test_block_backward(m, T, over, off):
    cfg, layer, x, resid, w, dout = problem(m, T, 5, **over)
    layer.cfg.route_scale = over.get("route_scale", 1.0)
    H, I, Nr, Kr, Ns = cfg["H"], cfg["I"], cfg["Nr"], cfg["Kr"], cfg.get("Ns", 1)
    _, saved = layer.block_forward(x, resid, w, EPS)
    bal = None
    if off is not None:
        offd = torch.tensor(off, dtype=torch.int32).cuda()
        loss, bal = layer.balance_loss(T, offd, alpha=5.0)
        bal["dloss"] = torch.randn(len(off) - 1, generator=torch.Generator().manual_seed(1)).cuda()
    g = layer.block_backward(saved, dout, balance=bal, dx_dtype=torch.float32)
    layer.check()
    # the experts' weight gradients, bit for bit those of the layer's own backward
    bws, BL = layer.block_backward_workspace(T), m.moe_backward_workspace_layout(layer.cfg, T)
    R, RS = T * Kr, T * (Kr + Ns)

    def view(name, shape):
        o, _ = BL[name]
        n = int(np.prod(shape))
        return bws[o:o + 4 * n].view(torch.float32).view(shape).cpu().double().numpy()

    GU, dh, dxr = view("gu", (RS, 2 * I)), view("dh", (RS, I)), view("dx_rows", (RS, H))
    _, dW13, dW2 = layer.backward(saved["y"], dout)
    assert torch.equal(g["dW13"], dW13) and torch.equal(g["dW2"], dW2)
    # the router: g dL/dg of each slot from the call's dh and h, the loss, and the two products
    ws, L = layer.workspace(T), layer.layout(T)
    pos = m.ws_view(ws, L, "pos", torch.int32, (T, Kr)).cpu().numpy().astype(np.int64)
    gate = f64(m.ws_view(ws, L, "gate", torch.float32, (T, Kr)))
    logits, idx = layer.router_state(T)
    idn, z = idx.cpu().numpy().astype(np.int64), f64(logits).sum(0)
    G, Uu = GU[:, :I], GU[:, I:]
    sg, _ = O.sigmoid(G)
    terms = dh * (G * sg * Uu)
    a = terms.sum(1)[pos]
    rs = layer.cfg.route_scale
    if bal is not None:
        lr, cr = O.balance_loss(z, idn, off, 5.0)
        assert np.array_equal(bal["counts"].cpu().numpy(), cr)
        assert (np.abs(f64(loss) - lr) <= 1e-5 * lr).all()
    kw = {} if bal is None else dict(off=off, counts=cr, dloss=bal["dloss"].cpu().numpy(), alpha=5.0)
    dz, mag = O.router_dlogits(z, idn, dgate=a / gate, route_scale=rs, **kw)
    # a itself: silu (expf, a quotient, products: 8), 128 terms in 4 + 5 steps, I / 128 shares; its magnitude is that of
    # the terms, not of their sum
    _, amag = O.router_dlogits(z, idn, dgate=np.abs(terms).sum(1)[pos] / gate, route_scale=rs)
    dz_err = (4 * z_tol(logits.cpu()) + 40 * U) * mag + (8 + 9 + I / 128) * U * amag
    wr, yy = f64(layer.wr), f64(saved["y"])
    Np, nt = (Nr + 63) // 64 * 64, (T + 31) // 32 * 32
    prod = (3 * max(Np, nt) / 16 + 150) * 4 * U
    assert (np.abs(f64(g["dwr"]) - dz.T @ yy) <= dz_err.T @ np.abs(yy) + prod * (np.abs(dz).T @ np.abs(yy))).all()
    # dy: the token's rows and the router's product, then the norm, and dout past it
    rows = dxr[pos].sum(1) + (dxr[R:] if Ns else 0)
    rmag = np.abs(dxr)[pos].sum(1) + (np.abs(dxr[R:]) if Ns else 0)
    dy = rows + dz @ wr
    dy_err = dz_err @ np.abs(wr) + prod * (np.abs(dz) @ np.abs(wr)) + (Kr + 2) * U * (rmag + np.abs(dz) @ np.abs(wr))
    ref, dn = O.rmsnorm_backward(dy, f64(saved["h"]), f64(saved["rstd"]), f64(w), f64(dout))
    n = f64(saved["h"]) * f64(saved["rstd"])[:, None]
    wd, r = np.abs(f64(w)), f64(saved["rstd"])[:, None]
    lin = lambda v: r * (v * wd + np.abs(n) * (v * wd * np.abs(n)).mean(1, keepdims=True))  # noqa: E731
    assert (np.abs(f64(g["dx"]) - ref) <= lin(dy_err) + 77 * U * (np.abs(f64(dout)) + lin(np.abs(dy)))).all()
    assert (np.abs(f64(g["dnorm"]) - dn) <= (dy_err * np.abs(n)).sum(0) + (T + 90) * U * (np.abs(dy) * np.abs(n)).sum(0)).all()
    # bf16 by default, and the same bits on every run
    g2 = layer.block_backward(saved, dout, balance=bal)
    assert torch.equal(g2["dx"], g["dx"].to(torch.bfloat16)) and torch.equal(g2["dwr"], g["dwr"])
    assert torch.equal(g2["dnorm"], g["dnorm"])


def test_block_step_captured(m):
    """A whole training step (forward, loss, backward) captured once and replayed on new inputs."""
    T = 160
    cfg, layer, x, resid, w, dout = problem(m, T, 7)
    off = torch.tensor([0, 64, 160], dtype=torch.int32).cuda()
    ins = [(x.clone(), dout.clone()), (x.flip(0).contiguous(), (dout * 0.5).contiguous())]

    def step():
        out, saved = layer.block_forward(x, resid, w, EPS)
        loss, bal = layer.balance_loss(T, off)
        g = layer.block_backward(saved, dout, balance=bal)
        return [out, loss] + [g[k] for k in ("dx", "dnorm", "dwr", "dW13", "dW2")]

    want = []
    for a, b in ins:
        x.copy_(a), dout.copy_(b)
        want.append([t.clone() for t in step()])
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        got = step()
    for (a, b), wnt in zip(ins, want):
        x.copy_(a), dout.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, wnt):
            assert torch.equal(p, q)
    layer.check()


def test_gate_gradient_against_the_unquantized_block(m):
    """dL/dg_k = FFN_k(y) . dout: the backward's g dL/dg, from its quantized dh and h, against the forward's gate-scaled
    expert outputs in the workspace.  The two carry the quantization of dout, h, W2's input and the FP32 sums
    differently: every E4M3 code is off by at most 2^-4 of itself, twice per term, so a slot differs by at most 2^-3 of
    the sum of its terms' magnitudes (and on the whole by far less)."""
    T = 200
    cfg, layer, x, resid, w, dout = problem(m, T, 11)
    H, I, Kr = cfg["H"], cfg["I"], cfg["Kr"]
    _, saved = layer.block_forward(x, resid, w, EPS)
    ws, L = layer.workspace(T), layer.layout(T)
    rows = f64(m.ws_view(ws, L, "y", torch.float32, (T * (Kr + 1), H)))
    pos = m.ws_view(ws, L, "pos", torch.int32, (T, Kr)).cpu().numpy().astype(np.int64)
    want = np.einsum("tkh,th->tk", rows[pos], f64(dout))
    layer.block_backward(saved, dout)
    bws, BL = layer.block_backward_workspace(T), m.moe_backward_workspace_layout(layer.cfg, T)

    def view(name, n):
        o, _ = BL[name]
        return bws[o:o + 4 * T * (Kr + 1) * n].view(torch.float32).view(-1, n).cpu().double().numpy()

    GU, dh = view("gu", 2 * I), view("dh", I)
    sg, _ = O.sigmoid(GU[:, :I])
    terms = dh * (GU[:, :I] * sg * GU[:, I:])
    got = terms.sum(1)[pos]
    # terms of the double sum over I and H: |h| |W2| |dout|; their l2 size bounds what independent roundings do
    assert np.linalg.norm(got - want) <= 2.0 ** -3 * np.linalg.norm(want)


def test_block_backward_captured_first_and_in_place(m):
    """A layer's first backward under capture, then an eager one before any replay: the transposed weights of the
    captured call are not there yet.  And bf16 dx in dout's, h's and y's place."""
    T = 96
    cfg, layer, x, resid, w, dout = problem(m, T, 11)
    out, saved = layer.block_forward(x, resid, w, EPS)
    layer.block_backward_workspace(T)
    torch.cuda.synchronize()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = layer.block_backward(saved, dout)
    want = {k: v.clone() for k, v in layer.block_backward(saved, dout).items()}
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    fresh = problem(m, T, 11)[1]
    fresh.block_forward(x, resid, w, EPS)
    ref = fresh.block_backward(saved, dout)
    assert all(torch.equal(ref[k], want[k]) for k in want)
    for name in ("dout", "h", "y"):
        a = dict(h=saved["h"].clone(), y=saved["y"].clone(), dout=dout.clone())
        r = m.moe_block_backward(layer.cfg, layer.weights(), layer._wt, a["h"], a["y"], saved["rstd"], a["dout"],
                                 layer.workspace(T), norm_weight=w, dx=a[name], err=layer.err)
        assert r[0] is a[name] and torch.equal(r[0], want["dx"]), name
    layer.check()

"""Operators around the MoE layer, as measured: residual addition + RMS norm + FP8 quantization and its
backward, the sequence-wise balance loss with its gradient, and the router's backward.

Each case names its operator under "op".  `run` with own = False is the plain
form in elementary torch operations; with own = True it makes the calls a user
of the package makes.
"""
import math

import torch

own = False

# The layer's model shape (hidden 7168, 256 routed experts, top-8) and the small parity shape (hidden 512, 16
# experts, top-4); token counts of decode, prefill and training batches.
V3 = dict(H=7168, Nr=256, Kr=8)
TINY = dict(H=512, Nr=16, Kr=4)
EPS = 1e-6
ALPHA = 1e-4


def listed():
    return [
        # one new token of one sequence: latency
        dict(name="norm_fwd_1_token", op="norm_fwd", T=1, H=7168, stream="bf16", resid=True, pow2=False),
        # a decode batch of 64
        dict(name="norm_fwd_decode_64", op="norm_fwd", T=64, H=7168, stream="bf16", resid=True, pow2=False),
        # a prefill or training batch
        dict(name="norm_fwd_4096", op="norm_fwd", T=4096, H=7168, stream="bf16", resid=True, pow2=False),
        # a long batch with the residual stream kept in FP32 and power-of-two scales
        dict(name="norm_fwd_16384_f32", op="norm_fwd", T=16384, H=7168, stream="f32", resid=True, pow2=True),
        # an odd number of tokens of a small model, gradients in bf16
        dict(name="norm_bwd_509_small", op="norm_bwd", T=509, H=512, stream="bf16", dy="bf16", dx="bf16"),
        # a training batch: the layer's FP32 input gradient back into a bf16 residual stream
        dict(name="norm_bwd_4096", op="norm_bwd", T=4096, H=7168, stream="bf16", dy="f32", dx="bf16"),
        # a long training batch, FP32 throughout
        dict(name="norm_bwd_16384_f32", op="norm_bwd", T=16384, H=7168, stream="f32", dy="f32", dx="f32"),
        # a few short packed sequences of the small router
        dict(name="balance_300_small", op="balance", T=300, Nr=16, Kr=4, S=8, n_seq=5),
        # packed sequences of many lengths in a long batch, with padding behind the last
        dict(name="balance_16384", op="balance", T=16384, Nr=256, Kr=8, S=1, n_seq=13),
        # the small router's gradients
        dict(name="router_bwd_256_small", op="router_bwd", T=256, H=512, Nr=16, Kr=4, S=8, n_seq=2),
        # a training batch
        dict(name="router_bwd_4096", op="router_bwd", T=4096, H=7168, Nr=256, Kr=8, S=2, n_seq=4),
        # a long one, an odd number of tokens
        dict(name="router_bwd_16381", op="router_bwd", T=16381, H=7168, Nr=256, Kr=8, S=1, n_seq=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance", "router_bwd"])
    T = _log_int(rng, 1, 16384)
    H = 128 * _log_int(rng, 1, 56)
    Nr = _log_int(rng, 4, 256)
    Kr = rng.randint(1, min(8, Nr))
    if op == "norm_fwd":
        return dict(op=op, T=T, H=H, stream=rng.choice(["bf16", "f32"]), resid=rng.random() < 0.75,
                    pow2=rng.random() < 0.5)
    if op == "norm_bwd":
        return dict(op=op, T=T, H=H, stream=rng.choice(["bf16", "f32"]), dy=rng.choice(["bf16", "f32"]),
                    dx=rng.choice(["bf16", "f32"]))
    S = max(1, min(16, 148 // (((T + 127) // 128) * ((Nr + 127) // 128))))
    c = dict(op=op, T=T, Nr=Nr, Kr=Kr, S=min(S, 2 * H // 128), n_seq=rng.randint(1, max(1, min(T, 16))))
    if op == "router_bwd":
        c["H"] = H
    return c


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T = case["op"], case["T"]

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    st = dict(case=case)
    if op in ("norm_fwd", "norm_bwd"):
        H = case["H"]
        stream = _dt(case["stream"])
        st["w"] = 1.0 + randn(H, std=0.1)
        if op == "norm_fwd":
            st["x"] = randn(T, H, std=0.5, dtype=stream)
            st["resid"] = randn(T, H, std=2.0, dtype=stream) if case["resid"] else None
            # a user's program keeps its output buffers
            st["h"] = torch.empty_like(st["x"]) if case["resid"] else None
            st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            st["q"] = torch.empty((T, H), dtype=torch.uint8, device="cuda")
            st["s"] = torch.empty((T, H // 128), dtype=torch.float32, device="cuda")
            st["rstd"] = torch.empty((T,), dtype=torch.float32, device="cuda")
        else:
            st["h"] = randn(T, H, std=2.0, dtype=stream)
            st["rstd"] = (st["h"].double().square().mean(dim=1) + EPS).rsqrt().float()
            st["dy"] = randn(T, H, std=1e-2, dtype=_dt(case["dy"]))
            st["dres"] = randn(T, H, std=1e-2, dtype=stream)
            st["dx"] = torch.empty((T, H), dtype=_dt(case["dx"]), device="cuda")
            st["dw"] = torch.empty((H,), dtype=torch.float32, device="cuda")
        return st

    Nr, Kr, S, n_seq = case["Nr"], case["Kr"], case["S"], case["n_seq"]
    # router logits as the router leaves them: one partial per split of its contraction (std 0.02 sqrt(7168) in all)
    st["logits"] = randn(S, T, Nr, std=1.7 / math.sqrt(S))
    bias = (torch.rand((Nr,), generator=g, device="cuda") * 2 - 1) * 0.01
    st["idx"] = (torch.sigmoid(st["logits"].sum(0)) + bias).topk(Kr, dim=1).indices.to(torch.int32)
    # packed sequences: random cuts, possibly equal (an empty sequence), and padding tokens behind the last
    cuts = torch.rand((n_seq,), generator=g, device="cuda") * (T + 1)
    off = torch.cat([torch.zeros(1, device="cuda"), cuts.sort().values.floor()]).clamp(max=T)
    off[-1] = max(1, T - T // 50)
    st["off"] = torch.minimum(off, off[-1]).to(torch.int32)
    st["dloss"] = torch.rand((n_seq,), generator=g, device="cuda") + 0.5
    st["loss"] = torch.empty((n_seq,), dtype=torch.float32, device="cuda")
    st["counts"] = torch.empty((n_seq, Nr), dtype=torch.int32, device="cuda")
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "balance":
        st["dlogits"] = torch.empty((T, Nr), dtype=torch.float32, device="cuda")
    else:
        H = case["H"]
        st["x"] = randn(T, H, dtype=torch.bfloat16)
        st["wr"] = randn(Nr, H, std=0.02, dtype=torch.bfloat16)
        st["dgate"] = randn(T, Kr, std=1e-2)
        # the loss's forward has run: its counts are in hand
        st["counts"].copy_(_seq_counts(st["idx"], st["off"], T, Nr))
        st["dx"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
        st["dwr"] = torch.empty((Nr, H), dtype=torch.float32, device="cuda")
    return st


# ------------------------------------------------------------ plain forms
def _members(off, T):
    """[n_seq, T] in 64 bits: 1 where the token belongs to the sequence."""
    t = torch.arange(T, device=off.device)
    return ((t >= off[:-1, None]) & (t < off[1:, None])).double()


def _seq_counts(idx, off, T, Nr):
    picks = torch.zeros((T, Nr), dtype=torch.float64, device=idx.device)
    picks.scatter_add_(1, idx.long(), torch.ones_like(idx, dtype=torch.float64))
    return (_members(off, T) @ picks).to(torch.int32)


def _norm_fwd(st):
    c = st["case"]
    T, H = c["T"], c["H"]
    h = st["x"] if st["resid"] is None else (st["x"].float() + st["resid"].float()).to(st["x"].dtype)
    h32 = h.float()
    rstd = (h32.square().mean(dim=1) + EPS).rsqrt()
    y = h32 * rstd[:, None] * st["w"]
    tiles = y.view(T, H // 128, 128)
    amax = tiles.abs().amax(dim=2)
    if c["pow2"]:
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
        s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int()), torch.zeros_like(amax))
    else:
        s = amax / 448.0
    q = torch.where(s[:, :, None] > 0, tiles / s[:, :, None], torch.zeros_like(tiles)).clamp(-448, 448)
    return dict(h=h, y=y.to(torch.bfloat16), q=q.view(T, H).to(torch.float8_e4m3fn), s=s, rstd=rstd)


def _norm_bwd(st):
    dy, h, dres = st["dy"].float(), st["h"].float(), st["dres"].float()
    r = st["rstd"][:, None]
    n = h * r
    gy = dy * st["w"]
    dx = dres + r * (gy - n * (gy * n).mean(dim=1, keepdim=True))
    return dict(dx=dx.to(st["dx"].dtype), dw=(dy * n).sum(dim=0))


def _affinity(logits):
    z = logits.sum(0)
    return torch.sigmoid(z), torch.sigmoid(-z)  # s and 1 - s


def _token_seq(off, T):
    t = torch.arange(T, device=off.device, dtype=torch.int32)
    seq = torch.searchsorted(off, t, right=True) - 1  # the last sequence that starts at or before t
    inside = (seq >= 0) & (seq < off.numel() - 1)
    return seq.clamp(0, off.numel() - 2), inside


def _balance(st, s, counts):
    Nr, Kr = st["case"]["Nr"], st["case"]["Kr"]
    o = st["off"].long()
    L = (o[1:] - o[:-1]).clamp(min=1).float()
    p = s / s.sum(dim=1, keepdim=True)
    mean_p = (_members(st["off"], st["case"]["T"]) @ p.double()).float() / L[:, None]
    f = counts.float() * (Nr / (Kr * L))[:, None]
    return ALPHA * (f * mean_p).sum(dim=1), f, L, p


def _balance_grad(st, s, om, counts):
    _, f, L, p = _balance(st, s, counts)
    seq, inside = _token_seq(st["off"], st["case"]["T"])
    ft = f[seq]
    k = torch.where(inside, st["dloss"][seq] * ALPHA / L[seq], torch.zeros_like(L[seq]))[:, None]
    return k * (p * om) * (ft - (ft * p).sum(dim=1, keepdim=True))


def _run_balance(st):
    s, om = _affinity(st["logits"])
    counts = _seq_counts(st["idx"], st["off"], st["case"]["T"], st["case"]["Nr"])
    return dict(loss=_balance(st, s, counts)[0], counts=counts, dlogits=_balance_grad(st, s, om, counts))


def _run_router_bwd(st):
    s, om = _affinity(st["logits"])
    dz = _balance_grad(st, s, om, st["counts"])
    i = st["idx"].long()
    ss = s.gather(1, i)
    gh = ss / ss.sum(dim=1, keepdim=True)
    dgate = st["dgate"]
    dz = dz.scatter_add(1, i, om.gather(1, i) * gh * (dgate - (dgate * gh).sum(dim=1, keepdim=True)))
    return dict(dx=dz @ st["wr"].float(), dwr=dz.t() @ st["x"].float())


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return dict(norm_fwd=_norm_fwd, norm_bwd=_norm_bwd, balance=_run_balance, router_bwd=_run_router_bwd)[op](state)


# ------------------------------------------------------ the package's calls
def _own(st):
    import sparse_moe_layer_expert_b200 as M
    c = st["case"]
    op = c["op"]
    if op == "norm_fwd":
        h, y, q, s, rstd = M.fp8_add_rmsnorm_quant_1x128(st["x"], st["resid"], st["w"], EPS, h=st["h"], y=st["y"],
                                                         q=st["q"], scales=st["s"], rstd=st["rstd"], pow2=c["pow2"])
        return dict(h=h, y=y, q=q.view(torch.float8_e4m3fn), s=s, rstd=rstd)
    if op == "norm_bwd":
        dx, dw = M.add_rmsnorm_backward(st["dy"], st["h"], st["rstd"], st["w"], dres=st["dres"], dx=st["dx"],
                                        dw=st["dw"])
        return dict(dx=dx, dw=dw)
    cfg = M.config(c.get("H", 128), 128, c["Nr"], c["Kr"])
    bal = dict(seq_offsets=st["off"], counts=st["counts"], dloss=st["dloss"], alpha=ALPHA)
    if op == "balance":
        loss, counts = M.moe_balance_loss(cfg, st["logits"], st["idx"], st["off"], alpha=ALPHA, loss=st["loss"],
                                          counts=st["counts"], err=st["err"])
        dlogits, _, _ = M.moe_router_backward(cfg, st["logits"], st["idx"], balance=bal, dlogits=st["dlogits"],
                                              err=st["err"])
        return dict(loss=loss, counts=counts, dlogits=dlogits)
    _, dx, dwr = M.moe_router_backward(cfg, st["logits"], st["idx"], x=st["x"], wr=st["wr"], dgate=st["dgate"],
                                       balance=bal, dx=st["dx"], dwr=st["dwr"], err=st["err"])
    return dict(dx=dx, dwr=dwr)


# --------------------------------------------------------------- the work
def work(case):
    op, T = case["op"], case["T"]
    if op == "norm_fwd":
        H, e = case["H"], 2 if case["stream"] == "bf16" else 4
        n = T * H
        return {"bytes": n * (e * (3 if case["resid"] else 1) + 2 + 1) + T * (H // 128) * 4 + T * 4 + H * 4,
                "flops": 8 * n}
    if op == "norm_bwd":
        H, e = case["H"], 2 if case["stream"] == "bf16" else 4
        n = T * H
        return {"bytes": n * (2 * e + (2 if case["dy"] == "bf16" else 4) + (2 if case["dx"] == "bf16" else 4)) +
                T * 4 + 2 * H * 4, "flops": 10 * n}
    Nr, Kr, S, n_seq = case["Nr"], case["Kr"], case["S"], case["n_seq"]
    state = S * T * Nr * 4 + T * Kr * 4 + (n_seq + 1) * 4
    if op == "balance":
        return {"bytes": state + T * Nr * 4 + n_seq * (Nr * 4 + 8), "flops": (S + 20) * T * Nr}
    H = case["H"]
    return {"bytes": state + T * Kr * 4 + n_seq * (Nr * 4 + 4) + T * H * (2 + 4) + Nr * H * (2 + 4),
            "flops": 4 * T * Nr * H + (S + 20) * T * Nr}


# ------------------------------------------------------- 64-bit definitions
def _e4m3(v):
    """The nearest E4M3 value of |v| <= 448 (ties to even), in 64 bits."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * torch.round(a / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    D = torch.float64
    if op == "norm_fwd":
        H = case["H"]
        h = st["x"].to(D)
        if st["resid"] is not None:
            h = (h + st["resid"].to(D)).to(_dt(case["stream"])).to(D)  # the residual stream is held in its type
        rstd = 1.0 / torch.sqrt((h * h).sum(1) / H + EPS)
        y = torch.einsum("th,t,h->th", h, rstd, st["w"].to(D))
        amax = y.abs().view(T, -1, 128).max(2).values
        if case["pow2"]:
            s = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / 448))), torch.zeros_like(amax))
        else:
            s = amax / 448
        sc = s.repeat_interleave(128, 1)
        q = torch.where(sc > 0, _e4m3(y / sc.clamp(min=1e-300)), torch.zeros_like(y))
        return dict(h=h, y=y, q=q, s=s, rstd=rstd)
    if op == "norm_bwd":
        h, w = st["h"].to(D).requires_grad_(), st["w"].to(D).requires_grad_()
        # d/dh of sum dy h w / rms(h), with the saved 1/rms as its value and eps from it
        eps = 1.0 / st["rstd"].to(D) ** 2 - h.detach().square().mean(1)
        y = h * w / torch.sqrt(h.square().mean(1) + eps)[:, None]
        dx, dw = torch.autograd.grad(y, (h, w), st["dy"].to(D))
        return dict(dx=dx + st["dres"].to(D), dw=dw)
    Nr, Kr = case["Nr"], case["Kr"]
    z = st["logits"].to(D).sum(0).requires_grad_()
    s = 1.0 / (1.0 + torch.exp(-z))
    i = st["idx"].long()
    onehot = torch.zeros((T, Nr), dtype=D, device="cuda").scatter_(1, i, 1.0)
    losses, counts = [], []
    bounds = st["off"].tolist()
    p = s / s.sum(1, keepdim=True)
    for a, b in zip(bounds[:-1], bounds[1:]):
        c = onehot[a:b].sum(0)
        counts.append(c)
        losses.append(ALPHA * (c * Nr / (Kr * max(b - a, 1)) * p[a:b].sum(0) / max(b - a, 1)).sum())
    loss = torch.stack(losses)
    total = (loss * st["dloss"].to(D)).sum()
    if op == "balance":
        (dz,) = torch.autograd.grad(total, z)
        return dict(loss=loss.detach(), counts=torch.stack(counts).to(torch.int32), dlogits=dz)
    sel = s.gather(1, i)
    total = total + (sel / sel.sum(1, keepdim=True) * st["dgate"].to(D)).sum()
    (dz,) = torch.autograd.grad(total, z)
    return dict(dx=dz @ st["wr"].to(D), dwr=dz.t() @ st["x"].to(D))

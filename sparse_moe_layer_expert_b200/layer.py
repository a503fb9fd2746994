"""MoeLayer: device-resident weights, bias, workspace and error flag of one
FP8 DeepSeekMoE layer, with forward / bias-update calls into libmoefp8.

Plumbing only: torch allocates the buffers; quantization, routing, the
grouped GEMMs and the combine all run in the library's kernels.
"""
from __future__ import annotations

import contextlib

import torch

from . import _binding as B


class MoeLayer:
    def __init__(self, shape: dict, device="cuda"):
        """shape: dict with H, I, Nr, Kr and optionally Ns (1), n_groups,
        topk_groups, route_scale."""
        self.shape = dict(shape)
        self.cfg = B.config_from(shape)
        c = self.cfg
        self.E = c.n_routed + c.n_shared
        H, I = c.hidden, c.inter
        dev = torch.device(device)
        self.device = dev
        self.w13 = torch.empty((self.E, 2 * I, H), dtype=torch.uint8, device=dev)
        self.s13 = torch.empty((self.E, 2 * I // 128, H // 128), dtype=torch.float32, device=dev)
        self.w2 = torch.empty((self.E, H, I), dtype=torch.uint8, device=dev)
        self.s2 = torch.empty((self.E, H // 128, I // 128), dtype=torch.float32, device=dev)
        self.wr = torch.empty((c.n_routed, H), dtype=torch.bfloat16, device=dev)
        self.bias = torch.zeros((c.n_routed,), dtype=torch.float32, device=dev)
        self.err = B.new_err_flag(dev)
        self._ws: dict[int, torch.Tensor] = {}
        self._copies: dict = {}

    # -------------------------------------------------------------- weights
    def set_expert(self, e: int, w13_bf16: torch.Tensor, w2_bf16: torch.Tensor, stream=None) -> None:
        """Quantize expert e's bf16 weights (128x128 blocks) into place, with
        the scale rule of the layer's scale mode.  The transposed copies that
        the backward reads, where they exist, follow in the same call."""
        pow2 = self.cfg.scale_mode == B.MOE_SCALE_POW2
        B.fp8_quant_128x128(w13_bf16.contiguous(), q=self.w13[e], scales=self.s13[e], stream=stream, pow2=pow2)
        B.fp8_quant_128x128(w2_bf16.contiguous(), q=self.w2[e], scales=self.s2[e], stream=stream, pow2=pow2)
        wt = self._wt
        if wt is not None:
            first = range(self.E)[e]  # e may count from the end
            one = slice(first, first + 1)
            B.moe_transpose_weights(B.config(self.cfg.hidden, self.cfg.inter, 1, 1, 0),
                                    {k: t if k == "wr" else t[one] for k, t in self.weights().items()},
                                    out={k: t[one] for k, t in wt.items()}, stream=stream)

    def weights_changed(self, stream=None) -> None:
        """To be called after w13, s13, w2 or s2 were written in place other
        than by set_expert of this layer or a sibling: brings the transposed
        copies that the backward reads, where they exist, up to date."""
        wt = self._wt
        if wt is not None:
            B.moe_transpose_weights(self.cfg, self.weights(), out=wt, stream=stream)

    def set_router(self, wr_bf16: torch.Tensor, bias: torch.Tensor) -> None:
        self.wr.copy_(wr_bf16)
        self.bias.copy_(bias)

    @classmethod
    def from_generator(cls, shape: dict, expert_fn, wr: torch.Tensor, bias: torch.Tensor, device="cuda"):
        """expert_fn(e) -> (w13 bf16 [2I, H], w2 bf16 [H, I]) on `device`,
        called once per expert (routed 0..Nr-1, then shared)."""
        layer = cls(shape, device)
        for e in range(layer.E):
            w13, w2 = expert_fn(e)
            layer.set_expert(e, w13, w2)
            del w13, w2
        layer.set_router(wr, bias)
        return layer

    def sibling(self, bias: torch.Tensor | None = None, **shape_overrides) -> "MoeLayer":
        """A layer on the same device-resident weights with another routing
        configuration (e.g. n_groups, topk_groups) and bias; nothing is
        copied."""
        other = object.__new__(MoeLayer)
        other.shape = dict(self.shape, **shape_overrides)
        other.cfg = B.config_from(other.shape)
        other.E, other.device = self.E, self.device
        other.w13, other.s13, other.w2, other.s2, other.wr = self.w13, self.s13, self.w2, self.s2, self.wr
        other.bias = self.bias.clone() if bias is None else bias
        other.err = B.new_err_flag(self.device)
        other._ws = {}
        other._copies = self._copies
        return other

    def __getstate__(self) -> dict:
        # a copy of the layer makes transposed weights of its own
        return dict(self.__dict__, _copies={})

    def weights(self) -> dict:
        return dict(w13=self.w13, s13=self.s13, w2=self.w2, s2=self.s2, wr=self.wr)

    # -------------------------------------------------------------- forward
    # Guard bands (bytes, a multiple of 256) around every workspace, filled
    # with GUARD_BYTE and checked by check_guards(): a kernel writing past
    # either end of its workspace shows up there.  Off (0) unless set.
    guard_bytes = 0
    GUARD_BYTE = 0xA5

    def workspace(self, T: int) -> torch.Tensor:
        ws = self._ws.get(T)
        if ws is None:
            ws = self._ws[T] = self._scratch(B.moe_workspace_size(self.cfg, T))
        return ws

    def _scratch(self, nbytes: int) -> torch.Tensor:
        n, g = max(int(nbytes), 256), self.guard_bytes
        if not g:
            return torch.empty(n, dtype=torch.uint8, device=self.device)
        assert g % 256 == 0
        buf = torch.full((n + 2 * g,), self.GUARD_BYTE, dtype=torch.uint8, device=self.device)
        self._guarded = getattr(self, "_guarded", [])
        self._guarded.append((buf, g, n))
        return buf[g:g + n]

    # What a call allocates belongs to the stream it runs on; what it finds is
    # made known to the allocator as used there too, so that neither is given
    # away while that stream still works with it.
    def _on(self, stream):
        return contextlib.nullcontext() if stream is None else B._use_stream(stream, self.bias)

    def _used(self, t: torch.Tensor, stream=None) -> torch.Tensor:
        handle = torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else B._stream(stream)
        seen = t.__dict__.setdefault("on_streams", set())
        if handle not in seen:
            with self._on(stream):
                if not torch.cuda.is_current_stream_capturing():  # (a capture's memory has to outlive its graph anyway)
                    t.record_stream(torch.cuda.current_stream(t.device))
                    seen.add(handle)
        return t

    def check_guards(self) -> None:
        """Raise if any guard band around this layer's workspaces changed."""
        for buf, g, n in getattr(self, "_guarded", []):
            head, tail = buf[:g], buf[g + n:]
            if not (bool((head == self.GUARD_BYTE).all()) and bool((tail == self.GUARD_BYTE).all())):
                raise RuntimeError(f"workspace guard band overwritten (workspace of {n} bytes)")

    def forward(self, x: torch.Tensor, out=None, out_dtype=B.MOE_DTYPE_BF16, idx_out=None, counts_out=None,
                stream=None) -> torch.Tensor:
        T = x.shape[0]
        if stream is not None and (out is None or T not in self._ws):  # something is allocated
            with self._on(stream):
                return self.forward(x, out, out_dtype, idx_out, counts_out)
        return B.moe_forward(self.cfg, self.weights(), self.bias, x, out=out, out_dtype=out_dtype, idx_out=idx_out,
                             counts_out=counts_out, ws=self._used(self.workspace(T), stream), err=self.err,
                             stream=stream)

    def bias_update(self, counts: torch.Tensor, T: int, gamma: float = 0.001, stream=None) -> None:
        B.moe_bias_update(self.bias, counts, self.cfg.n_routed, T * self.cfg.top_k, gamma, stream=stream)

    def seq_balance_loss(self, T: int, seq_len: int, alpha: float = 1e-4, stream=None) -> torch.Tensor:
        """Sequence-wise balance loss of the batch of T tokens this layer's
        last forward of that size routed, one value per run of seq_len tokens."""
        return B.moe_seq_balance_loss(self.cfg, T, seq_len, self.workspace(T), self.err, alpha=alpha, stream=stream)

    def backward(self, x: torch.Tensor, dout: torch.Tensor, stream=None):
        """Gradients of the expert FFNs for the batch this layer's last forward
        of that size routed (routing held fixed): (dx, dW13, dW2) in FP32.
        The transposed weight copies the dgrad GEMMs read are made on first
        use and kept; set_expert and weights_changed bring them up to date."""
        T = x.shape[0]
        with self._on(stream):
            return B.moe_backward(self.cfg, self.weights(), self._transposed(), x, dout, self._used(self.workspace(T)),
                                  ws=self._used(self.backward_workspace(T)), err=self.err)

    # Transposed copies of the weights: one set for all siblings, in the same
    # memory from then on, so that a captured backward reads the weights as they
    # are when it is replayed.
    def _weight_tensors(self) -> tuple:
        return self.w13, self.s13, self.w2, self.s2

    @property
    def _wt(self) -> dict | None:
        c = self._copies
        # other tensors in the weights' places: the copies are not theirs
        if c and all(a is b for a, b in zip(c["of"], self._weight_tensors())):
            return c["wt"]
        return None

    def _transposed(self) -> dict:
        """The copies, made now if there are none, for the current stream."""
        cur = torch.cuda.current_stream(self.device)
        capturing = torch.cuda.is_current_stream_capturing()
        wt = self._wt
        if wt is None:
            wt = B.moe_transpose_weights(self.cfg, self.weights())
            # copies made while a graph is captured are filled when it is replayed: that graph's own
            if not capturing:
                if self._copies:
                    self._copies = {}
                self._copies.update(of=self._weight_tensors(), wt=wt, filled=cur.record_event(), on=cur)
        elif cur != self._copies["on"] and not capturing:
            # (a capture cannot wait for what runs outside it; torch.cuda.graph waits for the device first)
            cur.wait_event(self._copies["filled"])
        for t in wt.values():
            self._used(t)
        return wt

    def backward_workspace(self, T: int) -> torch.Tensor:
        bws = getattr(self, "_bws", None)
        if bws is None:
            bws = self._bws = {}
        ws = bws.get(T)
        if ws is None:
            ws = bws[T] = self._scratch(B.lib.moe_backward_workspace_size(B.ctypes_cfg(self.cfg), T))
        return ws

    # ---------------------------------------------- the block: norm + layer
    def block_forward(self, x: torch.Tensor, resid=None, norm_weight=None, eps: float = 1e-6, out=None,
                      out_dtype=B.MOE_DTYPE_BF16, idx_out=None, counts_out=None, stream=None):
        """h = x + resid, out = h + MoE(rmsnorm(h) * norm_weight): (out,
        saved).  `saved` is what block_backward takes; the routing and the
        experts' state stay in this layer's workspace for that batch size, so
        the backward has to come before its next forward of the same size."""
        with self._on(stream):
            out, h, y, rstd = B.moe_block_forward(self.cfg, self.weights(), self.bias, x, resid, norm_weight, eps,
                                                  out=out, out_dtype=out_dtype, idx_out=idx_out,
                                                  counts_out=counts_out, ws=self._used(self.workspace(x.shape[0])),
                                                  err=self.err)
        return out, dict(h=h, y=y, rstd=rstd, norm_weight=norm_weight)

    def router_state(self, T: int):
        """(logit partials [n_splits, T, N_r], picks [T, K_r]) that this
        layer's last forward of T tokens left in its workspace (views)."""
        L = self.layout(T)
        ws, Nr = self.workspace(T), self.cfg.n_routed
        n = L["logits"][1] // (T * Nr * 4) if T else 1
        return (B.ws_view(ws, L, "logits", torch.float32, (n, T, Nr)),
                B.ws_view(ws, L, "idx", torch.int32, (T, self.cfg.top_k)))

    def balance_loss(self, T: int, seq_offsets: torch.Tensor, alpha: float = 1e-4, stream=None):
        """Balance loss and per-expert counts of the packed sequences of the
        batch this layer's last forward of T tokens routed: (loss, grad), grad
        being what block_backward takes as `balance` (dloss: ones)."""
        logits, idx = self.router_state(T)
        with self._on(stream):
            self._used(self.workspace(T))
            loss, counts = B.moe_balance_loss(self.cfg, logits, idx, seq_offsets, alpha=alpha, err=self.err)
        return loss, dict(seq_offsets=seq_offsets, counts=counts, alpha=alpha)

    def block_backward(self, saved: dict, dout: torch.Tensor, balance=None, dx_dtype=None, stream=None) -> dict:
        """Gradients of block_forward's batch: dict(dx (of x and of resid),
        dnorm, dwr, dW13, dW2).  The weights are those of now: change them
        with set_expert, or call weights_changed."""
        T = dout.shape[0]
        with self._on(stream):
            g = B.moe_block_backward(self.cfg, self.weights(), self._transposed(), saved["h"], saved["y"],
                                     saved["rstd"], dout, self._used(self.workspace(T)),
                                     norm_weight=saved["norm_weight"], balance=balance, dx_dtype=dx_dtype,
                                     ws=self._used(self.block_backward_workspace(T)), err=self.err)
        return dict(zip(("dx", "dnorm", "dwr", "dW13", "dW2"), g))

    def block_backward_workspace(self, T: int) -> torch.Tensor:
        bws = getattr(self, "_bbws", None)
        if bws is None:
            bws = self._bbws = {}
        ws = bws.get(T)
        if ws is None:
            ws = bws[T] = self._scratch(B.lib.moe_block_backward_workspace_size(B.ctypes_cfg(self.cfg), T))
        return ws

    def check(self, stream=None) -> None:
        st, v = B.moe_check_device_error(self.err, stream)
        if st != B.MOE_OK:
            raise B.MoeError(st, f"device error flag {v:#x}")

    def layout(self, T: int) -> dict:
        return B.moe_workspace_layout(self.cfg, T)

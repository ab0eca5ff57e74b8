"""A padding-free MoE layer driven through libxmoe.

Owns every buffer of one layer invocation (allocated once, with torch, on the
GPU) and runs the forward and backward as the sequence of C-ABI calls the
X-MoE pages describe ("5.4 MoE模型在分布式训练中的应用", section 训练流程: gate,
dispatch, experts, combine, then the reverse path).  No arithmetic happens in
Python: every step is a libxmoe kernel.
"""
from __future__ import annotations

import functools
from typing import Dict

import torch

from . import (PFT, _on_device, mx8_scale_shape, xmoe_add_rmsnorm, xmoe_add_rmsnorm_bwd, xmoe_add_rmsnorm_bwd_workspace_size,
               xmoe_balance_loss, xmoe_balance_loss_workspace_size, xmoe_build_pft, xmoe_build_pft_shared,
               xmoe_build_pft_workspace_size, xmoe_combine,
               xmoe_combine_bwd, xmoe_dispatch_bwd, xmoe_expert_ffn_bwd,
               xmoe_expert_ffn_bwd_dact_gather, xmoe_expert_ffn_bwd_dw13_gather, xmoe_expert_ffn_bwd_dw2, xmoe_expert_ffn_bwd_dx,
               xmoe_expert_ffn_down, xmoe_expert_ffn_down_mx8, xmoe_expert_ffn_up, xmoe_expert_ffn_up_gather,
               xmoe_expert_ffn_up_mx8, xmoe_mx8_quantize_weights, xmoe_route, xmoe_route_bwd, xmoe_route_bwd_balance,
               xmoe_route_bwd_workspace_size, xmoe_route_workspace_size)


def _on_its_device(method):
    """The library launches on the current device: a layer's passes make its own the
    current one."""
    @functools.wraps(method)
    def run(self, *args, **kw):
        with _on_device(self.w["wg"]):
            return method(self, *args, **kw)
    return run


def _on(stream, device) -> torch.cuda.Stream:
    """The caller's stream (or its handle), or the current one of the device."""
    if stream is None:
        return torch.cuda.current_stream(device)
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _need(t, shape, dtypes, name: str, device) -> None:
    """What the calls of a pass would refuse, asked before its first launch: an
    exception between two launches leaves streams that nothing joins again."""
    if t is None:
        return
    if t.shape != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, the layer needs {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, the layer needs {dtypes[0]}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor on {device} is needed")


class _Written:
    """Orders what reads a layer's own copies of the weights, on any stream, behind
    what wrote them.  A capture neither records nor waits here (an event of one
    side of a capture cannot be waited for on the other): what a graph reads or
    writes is in the order in which it is captured and replayed."""

    def __init__(self):
        self.event, self.behind = None, set()

    @staticmethod
    def _capturing(stream) -> bool:
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def wrote(self, stream) -> None:
        if not self._capturing(stream):
            self.event, self.behind = torch.cuda.Event(), {stream.cuda_stream}
            self.event.record(stream)

    def read(self, stream) -> None:
        if self.event is not None and stream.cuda_stream not in self.behind and not self._capturing(stream):
            stream.wait_event(self.event)
            self.behind.add(stream.cuda_stream)


class PaddingFreeMoE:
    """Buffers and call sequence for one layer of T tokens.

    weights: dict with wg [d,E], w1/w3 [E,d,h], w2 [E,h,d]; optional shared-expert
    weights s1/s3 [d, n*h_s], s2 [n*h_s, d] (the shared experts side by side),
    logit_bias / select_bias fp32 [E].

    Neither pass materialises the expert-sorted copy of x: the gather is fused
    into the operand loads of the up-projection and of the weight gradient of
    W1/W3 (X-MoE article, section 2.1.2).  lean=True also drops the saved
    pre-activations H1/H3 and recomputes
    them in the backward (the same kernel, so bitwise the same values): what
    the backward needs from the forward shrinks to act, ye and the routing.

    Shared experts: a SwiGLU FFN of width n*h is the sum of n FFNs of width h
    over its column blocks.  When the shared width is a multiple of the routed
    h (and merge_shared), the shared experts become that many more experts that
    every token is routed to with weight 1: one buffer, one call per product
    for routed and shared experts together.  The layer then keeps the routed
    and shared weights in one [E + n, d, h] / [E + n, h, d] buffer, copied at
    construction and again by refresh_weights() (call it after changing the
    weights).  Otherwise (the default) the shared FFN runs as a separate
    FFN of its own width on a second stream beside the routed path.  Measured
    on the DeepSeek-MoE-16B shape the separate stream is ~2.7% faster: it fills
    the routed products' tails, and the merged buffer's mean rows per expert
    (routed and shared together) moves the down-projection and dA products to
    the smaller tile.

    balance_alpha > 0 adds the gate's balance loss: the forward leaves it in
    `loss` [1] and the per-expert slot counts in `counts` [n_seq, E] (its kernels
    run beside the experts), and the backward adds its gradient, times `dloss`,
    to the gate's.  n_seq sequences, whose tokens the forward's seq_offsets
    names (n_seq = 1: all tokens, or those it names)."""

    def __init__(self, weights: Dict[str, torch.Tensor], T: int, k: int, inv_tau: float = 1.0,
                 backward: bool = True, lean: bool = False, overlap: bool = True, merge_shared: bool = False,
                 balance_alpha: float = 0.0, n_seq: int = 1):
        self.w = weights
        wg, w1 = weights["wg"], weights["w1"]
        self.dtype = wg.dtype
        self.device = wg.device
        self.T, self.k, self.inv_tau = T, k, inv_tau
        self.d, self.E = wg.shape
        self.h = w1.shape[2]
        self.shared = weights.get("s1") is not None
        self.backward_enabled = backward
        self.lean = lean
        # overlap: the gate's backward and the routed weight gradients run on
        # streams of their own (default priority) beside the data gradients;
        # unmerged shared experts run on a second stream beside the routed path
        self.overlap = overlap
        dev, dt = self.device, self.dtype
        T, d, E, h = T, self.d, self.E, self.h
        self.hs = weights["s1"].shape[1] if self.shared else 0
        self.merged = self.shared and merge_shared and self.hs % h == 0
        self.ns = self.hs // h if self.merged else 0       # shared experts carried as routed ones
        Ec, kc = E + self.ns, k + self.ns                   # experts and slots per token in the buffer
        self.Ec, self.kc = Ec, kc
        R = T * kc
        self.R = R
        # dW1/dW3 beside dA and dX on the caller's stream when experts are
        # small (mean rows per expert <= 1024), else on the weight-gradient
        # stream after dW2.  Whole steps: DeepSeek-MoE-16B shape -1.0%,
        # Zipf-skewed -4%, long batch (1638 rows per expert) +0.4%.
        self.dw13_main = R <= 1024 * Ec
        self.written = _Written()
        if self.merged:
            self.W1 = torch.empty((Ec, d, h), dtype=dt, device=dev)
            self.W3 = torch.empty((Ec, d, h), dtype=dt, device=dev)
            self.W2 = torch.empty((Ec, h, d), dtype=dt, device=dev)
            self.refresh_weights()
        else:
            self.W1, self.W3, self.W2 = w1, weights["w3"], weights["w2"]
        self.wside = torch.cuda.Stream(device=dev) if backward else None
        self.gside = torch.cuda.Stream(device=dev) if backward else None
        f32 = dict(dtype=torch.float32, device=dev)
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), **f32)
        self.logits = torch.empty((T, E), **f32)
        self.pft = PFT(T, Ec, kc, dev)
        self.pft_ws = torch.empty(max(xmoe_build_pft_workspace_size(T, Ec, kc), 16), dtype=torch.uint8, device=dev)
        self.route_ws = torch.empty(max(xmoe_route_workspace_size(T, d, E, dt), 16), dtype=torch.uint8, device=dev)
        self.balance_alpha, self.n_seq = balance_alpha, n_seq
        if balance_alpha > 0:
            self.loss = torch.empty(1, **f32)
            self.counts = torch.empty((n_seq, E), dtype=torch.int32, device=dev)
            self.coef = torch.empty((n_seq, E), **f32)
            self.balance_ws = torch.empty(xmoe_balance_loss_workspace_size(T, E, n_seq), dtype=torch.uint8, device=dev)
        self.act = torch.empty((R, h), dtype=dt, device=dev)
        self.h13 = torch.empty((R, 2 * h), dtype=dt, device=dev) if backward else None
        self.ye = torch.empty((R, d), dtype=dt, device=dev)
        self.y = torch.empty((T, d), dtype=dt, device=dev)
        self.side_shared = self.shared and not self.merged
        if self.side_shared:
            hs = self.hs
            self.sh_off = torch.tensor([0, T], dtype=torch.int32, device=dev)
            self.sh_act = torch.empty((T, hs), dtype=dt, device=dev)
            self.sh_h13 = torch.empty((T, 2 * hs), dtype=dt, device=dev) if backward else None
            self.sh_y = torch.empty((T, d), dtype=dt, device=dev)
            self.side = torch.cuda.Stream(device=dev)
        if backward:
            self.dtopk_w_all = torch.empty((T, kc), **f32)  # every slot; the routed ones first
            self.dye = torch.empty((R, d), dtype=dt, device=dev)
            self.dh13 = torch.empty((R, 2 * h), dtype=dt, device=dev)
            self.dxs = torch.empty((R, d), dtype=dt, device=dev)
            self.dW1 = torch.empty((Ec, d, h), dtype=dt, device=dev)
            self.dW3 = torch.empty((Ec, d, h), dtype=dt, device=dev)
            self.dW2 = torch.empty((Ec, h, d), dtype=dt, device=dev)
            self.dx = torch.empty((T, d), dtype=dt, device=dev)
            self.dwg = torch.empty((d, E), **f32)
            self.rdx = torch.empty((T, d), dtype=dt, device=dev)  # the gate's term of dx
            self.rbwd_ws = torch.empty(max(xmoe_route_bwd_workspace_size(T, d, E, dt), 16), dtype=torch.uint8,
                                       device=dev)
            if self.side_shared:
                hs = self.hs
                self.sh_dh13 = torch.empty((T, 2 * hs), dtype=dt, device=dev)
                self.sh_dx = torch.empty((T, d), dtype=dt, device=dev)
                self._ds1 = torch.empty((1, d, hs), dtype=dt, device=dev)
                self._ds3 = torch.empty((1, d, hs), dtype=dt, device=dev)
                self._ds2 = torch.empty((1, hs, d), dtype=dt, device=dev)

    @_on_its_device
    def refresh_weights(self, stream=None) -> None:
        """Merged layout only: copy the routed and shared weights (the tensors in
        the weights dict, in their own layouts) into the layer's [E + n, ...]
        buffers, in place on `stream`.  The merged buffers are copies, so a
        caller that updates the weights (an optimizer step) calls this before
        the next forward; without merging the layer reads the caller's tensors
        directly and this does nothing.  Later passes wait for it, on whatever
        stream they are; the caller orders it behind passes that still read the
        old weights, if those are on other streams.  It allocates nothing, so it
        can sit inside a captured graph."""
        if not self.merged:
            return
        w, E, ns, d, h = self.w, self.E, self.ns, self.d, self.h
        main = _on(stream, self.device)
        with torch.cuda.stream(main):
            self.W1[:E].copy_(w["w1"])
            self.W3[:E].copy_(w["w3"])
            self.W2[:E].copy_(w["w2"])
            self.W1[E:].copy_(w["s1"].view(d, ns, h).permute(1, 0, 2))
            self.W3[E:].copy_(w["s3"].view(d, ns, h).permute(1, 0, 2))
            self.W2[E:].copy_(w["s2"].view(ns, h, d))
        self.written.wrote(main)

    # views of the unmerged shared-expert weights as a single expert of width n*h_s
    def _shared_w(self):
        w = self.w
        return w["s1"].unsqueeze(0), w["s3"].unsqueeze(0), w["s2"].unsqueeze(0)

    def _streams(self, stream):
        main = _on(stream, self.device)
        side = self.side if (self.side_shared and self.overlap) else main
        self.written.read(main)
        return main, side

    @_on_its_device
    def forward(self, x: torch.Tensor, stream=None, hook=None, probe=None, seq_offsets=None,
                token_mask=None) -> torch.Tensor:
        """seq_offsets int32 [n_seq + 1] and token_mask bool [T]: the tokens that the
        balance loss counts (None: one sequence, every token).  The backward
        reads them again.
        hook(name), if given, is called after each library call is enqueued.
        probe(name, stream), if given, is called right before and right after
        each up-projection launch ("up" / "up_end" for the routed experts,
        "shared_up" / "shared_up_end" for the shared ones) with the stream the
        launch goes to, e.g. to record events around it."""
        w = self.w
        mark = hook or (lambda name: None)
        around = probe or (lambda name, s: None)
        _need(x, (self.T, self.d), (self.dtype,), "x", self.device)
        if self.balance_alpha > 0:
            if self.n_seq > 1 and seq_offsets is None:
                raise ValueError("seq_offsets is required for more than one sequence")
            _need(seq_offsets, (self.n_seq + 1,), (torch.int32,), "seq_offsets", self.device)
            _need(token_mask, (self.T,), (torch.bool, torch.uint8), "token_mask", self.device)
        main, side = self._streams(stream)
        keep = self.backward_enabled and not self.lean
        if self.side_shared:
            side.wait_stream(main)
            s1, s3, s2 = self._shared_w()
            around("shared_up", side)
            xmoe_expert_ffn_up(x, s1, s3, self.sh_off, self.sh_act, h13=self.sh_h13 if keep else None, stream=side)
            around("shared_up_end", side)
            xmoe_expert_ffn_down(self.sh_act, s2, self.sh_off, self.sh_y, stream=side)
            if side is main:
                mark("shared_ffn")
        xmoe_route(x, w["wg"], self.k, self.topk_ids, self.topk_w, self.logits, self.inv_tau,
                   w.get("logit_bias"), w.get("select_bias"), workspace=self.route_ws, stream=main)
        mark("route")
        bs = main
        if self.balance_alpha > 0:
            self.seq_offsets, self.token_mask = seq_offsets, token_mask
            if self.overlap and self.gside is not None:
                bs = self.gside
                bs.wait_stream(main)
            xmoe_balance_loss(self.logits, self.topk_ids, self.balance_alpha, self.loss, self.counts, self.coef,
                              seq_offsets, token_mask, self.balance_ws, stream=bs)
            if bs is main:
                mark("balance_loss")
        if self.merged:
            xmoe_build_pft_shared(self.topk_ids, self.topk_w, self.E, self.ns, self.pft, self.pft_ws, stream=main)
        else:
            xmoe_build_pft(self.topk_ids, self.topk_w, self.E, self.pft, self.pft_ws, stream=main)
        mark("build_pft")
        around("up", main)
        xmoe_expert_ffn_up_gather(x, self.pft.token_ids, self.W1, self.W3, self.pft.expert_offsets, self.act,
                                  h13=self.h13 if keep else None, stream=main)
        around("up_end", main)
        xmoe_expert_ffn_down(self.act, self.W2, self.pft.expert_offsets, self.ye, stream=main)
        mark("expert_ffn")
        y_add = None
        if self.side_shared:
            main.wait_stream(side)
            y_add = self.sh_y
        xmoe_combine(self.ye, self.pft, self.T, self.y, y_add=y_add, stream=main)
        mark("combine")
        if bs is not main:
            main.wait_stream(bs)
        self.x = x
        return self.y

    @_on_its_device
    def backward(self, dy: torch.Tensor, stream=None, hook=None, dloss=None) -> torch.Tensor:
        """dloss: upstream gradient of the balance loss, fp32 [1] on the device
        (None: 1)."""
        w = self.w
        mark = hook or (lambda name: None)
        _need(dy, (self.T, self.d), (self.dtype,), "dy", self.device)
        if self.balance_alpha > 0:
            _need(dloss, (1,), (torch.float32,), "dloss", self.device)
        main, side = self._streams(stream)
        gs = self.gside if self.overlap else main
        dx_add = None
        if self.side_shared:
            side.wait_stream(main)
            s1, s3, s2 = self._shared_w()
            if self.lean:
                xmoe_expert_ffn_up(self.x, s1, s3, self.sh_off, None, self.sh_h13, stream=side)
                if side is main:
                    mark("recompute_shared_h13")
            xmoe_expert_ffn_bwd(self.x, s1, s3, s2, self.sh_act, self.sh_h13, dy, self.sh_off, self.sh_dh13,
                                self.sh_dx, self._ds1, self._ds3, self._ds2, stream=side)
            if side is main:
                mark("shared_ffn_bwd")
        off = self.pft.expert_offsets
        ws = self.wside if self.overlap else main
        # dA reads dy through the PFT and applies each row's combine weight
        # itself, so it does not wait for the combine backward, which runs
        # beside it on the weight-gradient stream: its dye feeds dW2 there and
        # its dtopk_w the gate's backward
        if ws is not main:
            ws.wait_stream(main)
        xmoe_combine_bwd(dy, self.ye, self.pft, self.dye, self.dtopk_w_all, stream=ws)
        if ws is main:
            mark("combine_bwd")
        # the gate's backward needs only the routed slots' dtopk_w, the logits
        # and x: it runs beside the expert backward.  With unmerged shared
        # experts it adds dz . wg^T into their dx; otherwise it writes its own
        # term, which the dispatch backward adds.
        rdst = self.sh_dx if self.side_shared else self.rdx
        if self.side_shared:
            gs = side
        if gs is not ws:
            gs.wait_stream(ws)
        if self.balance_alpha > 0:
            xmoe_route_bwd_balance(self.x, w["wg"], self.logits, self.topk_ids, self.dtopk_w, self.coef, rdst, self.dwg,
                                   self.rbwd_ws, self.inv_tau, accumulate=self.side_shared,
                                   seq_offsets=self.seq_offsets, token_mask=self.token_mask, dloss=dloss, stream=gs)
        else:
            xmoe_route_bwd(self.x, w["wg"], self.logits, self.topk_ids, self.dtopk_w, rdst, self.dwg,
                           self.rbwd_ws, self.inv_tau, accumulate=self.side_shared, stream=gs)
        if gs is main:
            mark("route_bwd")
        dx_add = rdst
        if self.lean:
            # recompute the pre-activations only (act is kept from the forward)
            xmoe_expert_ffn_up_gather(self.x, self.pft.token_ids, self.W1, self.W3, self.pft.expert_offsets,
                                      None, self.h13, stream=main)
            mark("recompute_h13")
        xmoe_expert_ffn_bwd_dact_gather(dy, self.pft.token_ids, self.pft.combine_weights, self.W2, self.h13, off,
                                        self.dh13, stream=main)
        mark("bwd_dact")
        # weight gradients: dW2 needs act and dye only; dW1/dW3 need dH1/dH3 and
        # the token rows, gathered through the PFT inside their loads
        xmoe_expert_ffn_bwd_dw2(self.act, self.dye, off, self.dW2, stream=ws)
        if ws is main:
            mark("bwd_dw2")
        w13 = main if self.dw13_main else ws
        if w13 is not main:
            w13.wait_stream(main)
        xmoe_expert_ffn_bwd_dw13_gather(self.x, self.pft.token_ids, self.dh13, off, self.dW1, self.dW3, stream=w13)
        if w13 is main:
            mark("bwd_dw13")
        xmoe_expert_ffn_bwd_dx(self.dh13, self.W1, self.W3, off, self.dxs, stream=main)
        mark("bwd_dx")
        main.wait_stream(gs)
        xmoe_dispatch_bwd(self.dxs, self.pft, self.T, self.dx, dx_add=dx_add, stream=main)
        mark("dispatch_bwd")
        # every gradient is complete in the caller's stream order (the gate's
        # stream joined before the dispatch backward); only streams this call
        # used are joined, so that the step can also be captured as a graph
        if ws is not main:
            main.wait_stream(ws)
        return self.dx

    def saved_bytes(self) -> int:
        """Bytes the backward needs from the forward (beyond x and the weights):
        routing results, the PFT, act and ye, plus H1/H3 unless lean."""
        def nb(t):
            return 0 if t is None else t.numel() * t.element_size()
        n = nb(self.topk_ids) + nb(self.topk_w) + nb(self.logits) + nb(self.act) + nb(self.ye)
        n += sum(nb(t) for t in self.pft.fields().values())
        if not self.lean:
            n += nb(self.h13)
        if self.side_shared:
            n += nb(self.sh_act) + (0 if self.lean else nb(self.sh_h13))
        return n

    # gradients in the layer's argument layout
    @property
    def dtopk_w(self) -> torch.Tensor:
        """[T, k] gradient of the routing weights (the routed slots)."""
        return self.dtopk_w_all[:, :self.k]

    @property
    def dw1(self) -> torch.Tensor:
        return self.dW1[:self.E]

    @property
    def dw3(self) -> torch.Tensor:
        return self.dW3[:self.E]

    @property
    def dw2(self) -> torch.Tensor:
        return self.dW2[:self.E]

    def _shared_grad(self, which: int) -> torch.Tensor:
        """[1, d, n*h_s] (ds1, ds3) or [1, n*h_s, d] (ds2)."""
        if not self.merged:
            return (self._ds1, self._ds3, self._ds2)[which]
        E, ns, d, h = self.E, self.ns, self.d, self.h
        if which == 2:
            return self.dW2[E:].reshape(1, ns * h, d)
        src = self.dW1 if which == 0 else self.dW3
        return src[E:].permute(1, 0, 2).reshape(1, d, ns * h)

    @property
    def ds1(self) -> torch.Tensor:
        return self._shared_grad(0)

    @property
    def ds3(self) -> torch.Tensor:
        return self._shared_grad(1)

    @property
    def ds2(self) -> torch.Tensor:
        return self._shared_grad(2)

    def grads(self) -> Dict[str, torch.Tensor]:
        g = {"dx": self.dx, "dwg": self.dwg, "dw1": self.dw1, "dw3": self.dw3, "dw2": self.dw2,
             "dtopk_w": self.dtopk_w, "dye": self.dye, "dxs": self.dxs, "dh13": self.dh13}
        if self.shared:
            g.update(ds1=self.ds1[0], ds3=self.ds3[0], ds2=self.ds2[0])
        return g


class MoEBlock:
    """Pre-norm and layer of a transformer block, for training:
      sum = x + residual;  y = rmsnorm(sum) * gamma;  out = layer(y)
    The caller's next block adds out to sum.  weights: the layer's, with "norm"
    (gamma [d]); the other arguments are PaddingFreeMoE's."""

    def __init__(self, weights: Dict[str, torch.Tensor], T: int, k: int, eps: float = 1e-6, **layer):
        self.moe = PaddingFreeMoE(weights, T, k, **layer)
        self.gamma, self.eps = weights["norm"], eps
        m = self.moe
        row = dict(dtype=m.dtype, device=m.device)
        self.sum = torch.empty((T, m.d), **row)
        self.y = torch.empty((T, m.d), **row)
        self.rstd = torch.empty(T, dtype=torch.float32, device=m.device)
        if m.backward_enabled:
            self.dx = torch.empty((T, m.d), **row)
            self.dgamma = torch.empty(m.d, dtype=torch.float32, device=m.device)
            self.ws = torch.empty(xmoe_add_rmsnorm_bwd_workspace_size(T, m.d, m.dtype), dtype=torch.uint8,
                                  device=m.device)

    def forward(self, x: torch.Tensor, residual=None, stream=None, **tokens):
        """(out, sum); tokens: the layer's seq_offsets and token_mask."""
        xmoe_add_rmsnorm(x, residual, self.gamma, self.eps, self.sum, self.y, rstd=self.rstd, stream=stream)
        return self.moe.forward(self.y, stream=stream, **tokens), self.sum

    def backward(self, dout: torch.Tensor, dsum=None, stream=None, dloss=None) -> torch.Tensor:
        """Gradient of x (and of residual) from those of out and sum; gamma's is in
        `dgamma`, the layer's where the layer leaves them."""
        dy = self.moe.backward(dout, stream=stream, dloss=dloss)
        xmoe_add_rmsnorm_bwd(dy, dsum, self.sum, self.gamma, self.rstd, self.dx, self.dgamma, self.ws, stream=stream)
        return self.dx


class MoEBlock8:
    """The same block for serving, its experts in 8 bits: the norm leaves y for the
    gate and y in 8 bits for the experts, whose weights are quantized once at
    construction (again by refresh_weights() after they change).  Weights as
    PaddingFreeMoE takes them, with "norm": the gate's and the norm's in bf16,
    the experts' in bf16 or fp32; d, h and the shared width multiples of 32.  Shared experts run on a second stream beside the routed
    ones.  Holds the buffers of T tokens."""

    def __init__(self, weights: Dict[str, torch.Tensor], T: int, k: int, inv_tau: float = 1.0, eps: float = 1e-6,
                 overlap: bool = True):
        self.w, self.T, self.k, self.inv_tau, self.eps, self.overlap = weights, T, k, inv_tau, eps, overlap
        wg, w1 = weights["wg"], weights["w1"]
        dev, dt = wg.device, wg.dtype
        for n in ("wg", "norm"):
            if weights[n].dtype != torch.bfloat16:
                raise TypeError(f"{n}: dtype {weights[n].dtype}, the block needs {torch.bfloat16}")
        self.device, (self.d, self.E), self.h = dev, wg.shape, w1.shape[2]
        d, E, h, R = self.d, self.E, self.h, T * k
        self.shared = weights.get("s1") is not None
        f8, u8 = dict(dtype=torch.float8_e4m3fn, device=dev), dict(dtype=torch.uint8, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)

        def rows(n, K):
            return torch.empty((n, K), **f8), torch.empty(mx8_scale_shape(n, K), **u8)

        def experts(n, N, K):
            return torch.empty((n, N, K), **f8), torch.empty((n,) + mx8_scale_shape(N, K), **u8)

        self.sum, self.y, self.out = (torch.empty((T, d), **bf) for _ in range(3))
        self.yq, self.yqs = rows(T, d)
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        self.pft = PFT(T, E, k, dev)
        self.pft_ws = torch.empty(max(xmoe_build_pft_workspace_size(T, E, k), 16), **u8)
        self.route_ws = torch.empty(max(xmoe_route_workspace_size(T, d, E, dt), 16), **u8)
        self.act, self.acts = rows(R, h)
        self.ye = torch.empty((R, d), **bf)
        self.w1q, self.w3q, self.w2q = experts(E, h, d), experts(E, h, d), experts(E, d, h)
        if self.shared:
            hs = weights["s1"].shape[1]
            self.s1q, self.s3q, self.s2q = experts(1, hs, d), experts(1, hs, d), experts(1, d, hs)
            self.sh_off = torch.tensor([0, T], dtype=torch.int32, device=dev)
            self.sh_act, self.sh_acts = rows(T, hs)
            self.sh_y = torch.empty((T, d), **bf)
            self.side = torch.cuda.Stream(device=dev)
        self.written = _Written()
        self.refresh_weights()

    @_on_its_device
    def refresh_weights(self, stream=None) -> None:
        """Quantize the weights (the tensors in the weights dict) again.  Later
        forwards wait for it, on whatever stream they are; the caller orders it
        behind the update of the weights and behind forwards that still read the
        old ones, if those are on other streams."""
        w = self.w
        stream = _on(stream, self.device)
        pairs = [(w["w1"], self.w1q), (w["w3"], self.w3q), (w["w2"], self.w2q)]
        if self.shared:
            pairs += [(w[n].unsqueeze(0), q) for n, q in (("s1", self.s1q), ("s3", self.s3q), ("s2", self.s2q))]
        for t, (q, s) in pairs:
            xmoe_mx8_quantize_weights(t, q, s, stream=stream)
        self.written.wrote(stream)

    @_on_its_device
    def forward(self, x: torch.Tensor, residual=None, stream=None):
        """(out, sum)."""
        w = self.w
        main = _on(stream, self.device)
        side = self.side if self.shared and self.overlap else main
        self.written.read(main)
        xmoe_add_rmsnorm(x, residual, w["norm"], self.eps, self.sum, self.y, self.yq, self.yqs, stream=main)
        if self.shared:
            if side is not main:
                side.wait_stream(main)
            xmoe_expert_ffn_up_mx8(self.yq, self.yqs, *self.s1q, *self.s3q, self.sh_off, self.sh_act, self.sh_acts,
                                   stream=side)
            xmoe_expert_ffn_down_mx8(self.sh_act, self.sh_acts, *self.s2q, self.sh_off, self.sh_y, stream=side)
        xmoe_route(self.y, w["wg"], self.k, self.topk_ids, self.topk_w, self.logits, self.inv_tau, w.get("logit_bias"),
                   w.get("select_bias"), workspace=self.route_ws, stream=main)
        xmoe_build_pft(self.topk_ids, self.topk_w, self.E, self.pft, self.pft_ws, stream=main)
        xmoe_expert_ffn_up_mx8(self.yq, self.yqs, *self.w1q, *self.w3q, self.pft.expert_offsets, self.act, self.acts,
                               token_ids=self.pft.token_ids, stream=main)
        xmoe_expert_ffn_down_mx8(self.act, self.acts, *self.w2q, self.pft.expert_offsets, self.ye, stream=main)
        if side is not main:
            main.wait_stream(side)
        xmoe_combine(self.ye, self.pft, self.T, self.out, y_add=self.sh_y if self.shared else None, stream=main)
        return self.out, self.sum

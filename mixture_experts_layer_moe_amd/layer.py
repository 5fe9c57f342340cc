"""One GPU's share of an MoE layer: the four library calls on preallocated buffers.

Marshalling only: buffers are allocated once with torch, and `run()` enqueues
moe_route_topk -> moe_permute -> moe_grouped_ffn -> moe_combine on one stream
with no host synchronisation in between (every data-dependent size stays on
the device), so the whole layer can also be captured in a HIP graph.  With
fused_gather=True the permute writes indices only and moe_grouped_ffn_gather
reads layer0's token rows straight from x (no x_perm).  With signalled=True
the grouped FFN and the combine run as one launch with tile-level signals
(moe_ffn_combine_fused; 256-row tiles).  With a Gating the tokens are routed
by moe_route_grouped instead of moe_route_topk; with a SharedExpert every token
also goes through a dense FFN (two moe_linear calls) whose down product is
added to the combined output.  With experts in MXFP4 (ffi.Mxfp4 weights) the
tokens, in permute(), and the activations are quantised too and the grouped FFN
is two moe_grouped_linear_mxfp4 calls; a SharedExpert in MXFP4 runs the same way
on moe_linear_mxfp4.  Activations are then rounded twice, to bf16 where the first
product stores them and from there to 4 bits.

With few_tokens=True, for at most 64 tokens, routing, experts and combine are one
moe_few_tokens call over bf16 or MXFP4 experts, whose activations stay in full
precision.  It is the faster form for one token (145 us instead of 156 over 256
bf16 experts of 7168 x 2048, 55 instead of 85 in MXFP4), and for a few more where
experts are small or few: to 16 tokens over 64 bf16 experts of 2048 x 1408, to 8
in MXFP4; to 4 over 8 bf16 experts of 4096 x 14336, to 2 in MXFP4.  Beyond that
the other form reads the weights faster (tile_m 16, or 64 where experts have more
than 16 tokens).
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import ffi
from .ffi import Mxfp4, Weight
from .workloads import MoEConfig


@dataclass
class Gating:
    """How moe_route_grouped chooses and weights the experts (see include/moe.h)."""
    bias: Optional[torch.Tensor] = None  # [E] fp32, added to the scores for the choice only
    score: str = "sigmoid"
    n_group: int = 1
    topk_group: int = 1
    group_top: int = 1
    scale: float = 1.0


@dataclass
class SharedExpert:
    """A dense FFN of the layer's activation that every token goes through (output-major; bf16, or all in MXFP4).

    Where several GPUs' outputs are summed (shares of the experts), one of them has it.
    """
    w0: Weight               # [F_s, H]: W_gate^T (SwiGLU) or W1^T (GELU)
    w0_up: Optional[Weight]  # [F_s, H]: W_up^T (SwiGLU only)
    w1: Weight               # [H, F_s]


def _all_mxfp4(what: str, *weights) -> bool:
    """Whether the weights are in MXFP4: all of them or none."""
    mx = {isinstance(w, Mxfp4) for w in weights if w is not None}
    if len(mx) > 1:
        raise ValueError(f"{what} must all be in MXFP4, or none")
    return mx == {True}


class MoELayer:
    def __init__(self, cfg: MoEConfig, x: torch.Tensor, logits: torch.Tensor,
                 src_rank: Optional[torch.Tensor], w0: Weight, w0_up: Optional[Weight],
                 w1: Weight, tile_m: Optional[int] = None, renormalize: bool = True,
                 fused_gather: bool = False, signalled: bool = False,
                 gating: Optional[Gating] = None, shared: Optional[SharedExpert] = None,
                 few_tokens: bool = False):
        self.mxfp4 = _all_mxfp4("the experts' weights", w0, w0_up, w1)
        if signalled and (self.mxfp4 or few_tokens):
            raise ValueError("signalled runs bf16 experts, and not the form for a few tokens")
        if few_tokens and (fused_gather or cfg.T > ffi.FEW_TOKENS):
            raise ValueError(f"few_tokens takes at most {ffi.FEW_TOKENS} tokens, and permutes none")
        if shared is not None:
            Fs = shared.w0.shape[0]
            if (shared.w0_up is not None) != (cfg.act == "swiglu"):
                raise ValueError("shared.w0_up belongs to a SwiGLU layer, and only to one")
            for n, t, shape in (("w0", shared.w0, (Fs, cfg.H)), ("w0_up", shared.w0_up, (Fs, cfg.H)),
                                ("w1", shared.w1, (cfg.H, Fs))):
                if t is not None and t.shape != shape:
                    raise ValueError(f"shared.{n} must have shape {shape}, got {tuple(t.shape)}")
            self.shared_mxfp4 = _all_mxfp4("the shared expert's weights", shared.w0, shared.w0_up, shared.w1)
        self.cfg = cfg
        self.gating, self.shared = gating, shared
        self.few_tokens = few_tokens
        self.fused_gather = fused_gather or self.mxfp4  # (quantised tokens are gathered by their product)
        self.signalled = signalled
        self.tile_m = tile_m or cfg.tile_m
        self.renormalize = renormalize
        self.x, self.logits, self.src_rank = x, logits, src_rank
        self.w0, self.w0_up, self.w1 = w0, w0_up, w1
        dev = x.device
        T, H, k, El = cfg.T, cfg.H, cfg.k, cfg.n_local
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.out = torch.empty((T, H), dtype=torch.float32, device=dev)
        if few_tokens:
            self.few_ws = ffi.alloc_few_tokens_workspace(T, k, cfg.F_loc, dev)
        else:
            self.perm = ffi.alloc_permuted(T, H, k, El, self.tile_m, dev, rows=not self.fused_gather)
            nbytes = ffi.permute_workspace_bytes(T, k, El, cfg.num_ranks)
            self.ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
            self.act_buf = torch.empty((self.perm.R_cap, cfg.F_loc), dtype=torch.bfloat16, device=dev)
            self.y_perm = torch.empty((self.perm.R_cap, H), dtype=torch.float32, device=dev)
            ffn_bytes = 0 if self.mxfp4 else ffi.grouped_ffn_workspace_bytes(self.tile_m, H)
            self.ffn_ws = torch.empty(ffn_bytes, dtype=torch.uint8, device=dev) if ffn_bytes else None
            self.fused_ws = ffi.alloc_fused_workspace(self.perm.tiles_cap, H, dev) if signalled else None
            if self.mxfp4:
                self.act_q = ffi.alloc_mxfp4(self.act_buf.shape, dev)
        quantized = (self.mxfp4 and not few_tokens) or (shared is not None and self.shared_mxfp4)
        self.x_q = ffi.alloc_mxfp4((T, H), dev) if quantized else None
        if shared is not None:
            self.shared_h = torch.empty((T, Fs), dtype=torch.bfloat16, device=dev)
            if self.shared_mxfp4:
                self.shared_q = ffi.alloc_mxfp4((T, Fs), dev)
            else:
                self.shared_ws = [ffi.alloc_linear_workspace(T, Fs, H, cfg.act, dev),
                                  ffi.alloc_linear_workspace(T, H, Fs, "none", dev)]

    @classmethod
    def from_inputs(cls, cfg: MoEConfig, inputs: dict, **kw) -> "MoELayer":
        return cls(cfg, inputs["x"], inputs["logits"], inputs["src_rank"], inputs["w0"],
                   inputs["w0_up"], inputs["w1"], **kw)

    def route(self, stream=None):
        g = self.gating
        if g is not None:
            ffi.moe_route_grouped(self.logits, self.cfg.k, bias=g.bias, score=g.score, n_group=g.n_group,
                                  topk_group=g.topk_group, group_top=g.group_top, renormalize=self.renormalize,
                                  scale=g.scale, topk_idx=self.topk_idx, topk_w=self.topk_w, stream=stream)
            return
        ffi.moe_route_topk(self.logits, self.cfg.k, self.renormalize, self.topk_idx, self.topk_w, stream)

    def permute(self, stream=None):
        """Rows by expert; for experts in MXFP4 indices only, and the tokens quantised."""
        c = self.cfg
        if self.mxfp4:
            self.quantize_tokens(stream)
        ffi.moe_permute(self.x, self.topk_idx, self.src_rank, c.E, c.expert_begin, c.n_local,
                        c.num_ranks, self.tile_m, out=self.perm, ws=self.ws, stream=stream,
                        copy_rows=not self.fused_gather)

    def quantize_tokens(self, stream=None):
        """The tokens in MXFP4, for experts or a shared expert in MXFP4."""
        ffi.moe_mxfp4_quantize(self.x, out=self.x_q, stream=stream)

    def ffn(self, stream=None):
        if self.mxfp4:
            # (All of act_buf is quantised, as only the device knows how many of its rows have tokens; the others, as they
            # lie, belong to no product.  An eighth of 64 experts, 16384 tokens of 8 choices: 121 us for 133112 rows, where
            # the 16523 that have tokens would take 14.)
            ffi.moe_grouped_linear_mxfp4(self.perm, self.x_q, self.w0, w_up=self.w0_up, act=self.cfg.act, gather=True,
                                         out=self.act_buf, stream=stream)
            ffi.moe_mxfp4_quantize(self.act_buf, out=self.act_q, stream=stream)
            ffi.moe_grouped_linear_mxfp4(self.perm, self.act_q, self.w1, out=self.y_perm, stream=stream)
        elif self.fused_gather:
            ffi.moe_grouped_ffn_gather(self.x, self.perm, self.w0, self.w0_up, self.w1, self.cfg.act,
                                       self.act_buf, self.y_perm, self.ffn_ws, stream, use_workspace=False)
        else:
            ffi.moe_grouped_ffn(self.perm, self.w0, self.w0_up, self.w1, self.cfg.act,
                                self.act_buf, self.y_perm, self.ffn_ws, stream, use_workspace=False)

    def combine(self, stream=None):
        ffi.moe_combine(self.y_perm, self.perm.inv_perm, self.topk_w, self.out, stream)

    def ffn_combine(self, stream=None):
        """The grouped FFN and the combine as one launch with tile-level signals."""
        ffi.moe_ffn_combine_fused(self.perm, self.w0, self.w0_up, self.w1, self.cfg.act, self.topk_w,
                                  self.fused_ws, self.act_buf, self.y_perm, self.out, stream)

    def shared_expert(self, stream=None):
        """The shared expert's FFN, added to the combined output."""
        s = self.shared
        if self.shared_mxfp4:
            if not self.mxfp4 or self.few_tokens:  # (else permute() has done it)
                self.quantize_tokens(stream)
            ffi.moe_linear_mxfp4(self.x_q, s.w0, w_up=s.w0_up, act=self.cfg.act, out=self.shared_h, stream=stream)
            ffi.moe_mxfp4_quantize(self.shared_h, out=self.shared_q, stream=stream)
            ffi.moe_linear_mxfp4(self.shared_q, s.w1, residual=self.out, out=self.out, stream=stream)
            return
        ffi.moe_linear(self.x, s.w0, w_up=s.w0_up, act=self.cfg.act, out=self.shared_h, ws=self.shared_ws[0],
                       stream=stream, use_workspace=False)
        ffi.moe_linear(self.shared_h, s.w1, residual=self.out, out=self.out, ws=self.shared_ws[1], stream=stream,
                       use_workspace=False)

    def few(self, stream=None):
        """Experts and combine, and the routing where no Gating does it, in one call for a few tokens."""
        c = self.cfg
        ffi.moe_few_tokens(self.x, self.w0, self.w0_up, self.w1, c.act, logits=None if self.gating else self.logits,
                           renormalize=self.renormalize, topk_idx=self.topk_idx, topk_w=self.topk_w,
                           expert_begin=c.expert_begin, num_experts=c.E, out=self.out, ws=self.few_ws, stream=stream)

    def run(self, stream=None) -> torch.Tensor:
        if self.few_tokens:
            if self.gating is not None:
                self.route(stream)
            self.few(stream)
        else:
            self.route(stream)
            self.permute(stream)
            if self.signalled:
                self.ffn_combine(stream)
            else:
                self.ffn(stream)
                self.combine(stream)
        if self.shared is not None:
            self.shared_expert(stream)
        return self.out

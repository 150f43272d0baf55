"""A pre-norm residual block around one MoE layer:  h' = h + delta,
y = MoE(LayerNorm(h')), and the block's result is h' + y.

The sum h' + y is left to whoever comes next: a following block takes ``y`` as
its ``delta`` and adds it inside its own norm, so a stack of blocks never makes a
pass over the stream for it.  ``MoEBlock`` owns nothing but the pieces it is
given (``norm.LayerNorm``, ``layer.MoELayer`` and, for serving,
``decode.MoEDecoder``) and computes nothing itself.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B
from .decode import MoEDecoder
from .layer import MoELayer
from .norm import LayerNorm


class BlockState(NamedTuple):
    """What ``forward`` leaves for ``backward`` (with the layer's workspace)."""
    h: torch.Tensor        # the normalised stream
    z: torch.Tensor        # the layer's input
    mean: torch.Tensor
    rstd: torch.Tensor


class MoEBlock:
    def __init__(self, norm: LayerNorm, layer: MoELayer):
        if norm.D != layer.cfg.D:
            raise ValueError(f"the norm has {norm.D} channels, the layer {layer.cfg.D}")
        want = torch.bfloat16 if layer.dtype == "bf16" else torch.float32
        if norm.z_type != want:
            raise ValueError(f"the norm writes {norm.z_type}, the layer reads {want}")
        if norm.device != layer.w_gate.device:
            raise ValueError(f"the norm is on {norm.device}, the layer on {layer.w_gate.device}")
        self.norm, self.layer = norm, layer
        self._decoder: Optional[MoEDecoder] = None

    def forward(self, h, delta=None):
        """(state, y) of the layer's T tokens: state.h is the stream h + delta
        (h itself without a delta), y [T, D] fp32 the layer's output."""
        if h.shape[0] != self.layer.cfg.T:
            raise ValueError(f"the layer was made for {self.layer.cfg.T} tokens, got {tuple(h.shape)}")
        r = self.norm.forward(h, delta)
        return BlockState(h if r.h is None else r.h, r.z, r.mean, r.rstd), self.layer.forward(r.z)

    def backward(self, state: BlockState, dout):
        """Gradient [T, D] fp32 at state.h (and so at the delta) from dout (fp32),
        the one at state.h + y.  The layer's and the norm's parameter gradients are
        left in their buffers.  The layer's workspace must still hold the state
        of this block's forward."""
        # before the layer's launches, which take plain addresses
        shape = (self.layer.cfg.T, self.norm.D)
        self.norm._rows("dout", dout, torch.float32, shape)
        self.norm._rows("state.z", state.z, self.norm.z_type, shape)
        dz = torch.empty_like(dout)
        self.layer.backward(state.z, dout, dz)
        return self.norm.backward(dz, state.h, state.mean, state.rstd, dres=dout).dx

    @property
    def decoder(self) -> MoEDecoder:
        """The few-token form of the layer, on the weights it trains (made on
        the first use, which is outside of any graph capture)."""
        d = self._decoder
        if d is None:
            la, c = self.layer, self.layer.cfg
            lp = la.dtype == "bf16"
            pick = lambda name: getattr(la, name + "_lp" if lp else name)  # noqa: E731
            name_of = lambda table, v: next(k for k, i in table.items() if i == v)  # noqa: E731
            d = self._decoder = MoEDecoder(
                la.w_gate, pick("w1"), pick("w2"), w3=pick("w3"), b1=la.b1, b2=la.b2, k=c.k,
                act=name_of(B.ACT, c.act), score=name_of(B.SCORE, c.score), n_groups=c.n_groups,
                topk_groups=c.topk_groups, group_score=name_of(B.GROUP_SCORE, c.group_score),
                logit_bias=la.logit_bias, corr_bias=la.corr_bias, n_shared=c.n_shared,
                ws1=pick("ws1"), ws3=pick("ws3"), ws2=pick("ws2"),
                capacity_factor=c.capacity_factor)
        return d

    def decode(self, h, delta=None):
        """(h', y) for a few tokens: h' = h + delta (h without one) and y [T, D] in
        the layer's type, the next block's delta.  Both are buffers of this
        block, which its next call overwrites."""
        r = self.norm.forward(h, delta, stats=False)
        return h if r.h is None else r.h, self.decoder.decode(r.z)

"""A pre-norm residual block around one MoE layer:  h' = h + delta,
y = MoE(LayerNorm(h')), and the block's result is h' + y.

The sum h' + y is left to whoever comes next: a following block takes ``y`` as
its ``delta`` and adds it inside its own norm, so a stack of blocks never makes a
pass over the stream for it.  ``MoEBlock`` owns nothing but the pieces it is
given (``norm.LayerNorm``, ``layer.MoELayer`` and, for serving,
``decode.MoEDecoder``) and computes nothing itself.  ``Q4Block`` is the block on 4-bit
expert weights, for serving.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B
from .decode import MoEDecoder
from .layer import MoELayer
from .norm import LayerNorm
from .q4_layer import Q4Layer


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

    def _served(self):
        """The layer's tensors that serving reads, by the decoder's names for them
        and the layer's own."""
        la, lp = self.layer, "_lp" if self.layer.dtype == "bf16" else ""
        own = dict(w_gate="w_gate", w1="w1" + lp, w3="w3" + lp, w2="w2" + lp, b1="b1", b2="b2",
                   logit_bias="logit_bias", corr_bias="corr_bias", ws1="ws1" + lp, ws3="ws3" + lp,
                   ws2="ws2" + lp)
        return {name: (attr, getattr(la, attr)) for name, attr in own.items()}

    @property
    def decoder(self) -> MoEDecoder:
        """The few-token form of the layer, on the weights it trains (made on
        the first use, which is outside of any graph capture).  It reads the
        storage that they had then: once a tensor of the layer has been replaced,
        rather than changed in place, this raises; make a new block."""
        d = self._decoder
        if d is None:
            c = self.layer.cfg
            name_of = lambda table, v: next(k for k, i in table.items() if i == v)  # noqa: E731
            served = self._served()
            d = self._decoder = MoEDecoder(
                **{name: t for name, (_, t) in served.items()}, k=c.k, act=name_of(B.ACT, c.act),
                score=name_of(B.SCORE, c.score), n_groups=c.n_groups, topk_groups=c.topk_groups,
                group_score=name_of(B.GROUP_SCORE, c.group_score), n_shared=c.n_shared,
                capacity_factor=c.capacity_factor)
            self._read = [(attr, None if t is None else t.data_ptr()) for attr, t in served.values()]
            return d
        for attr, at in self._read:
            t = getattr(self.layer, attr)
            if (None if t is None else t.data_ptr()) != at:
                raise ValueError(f"the layer's {attr} was replaced after the decoder was made")
        return d

    def decode(self, h, delta=None):
        """(h', y) for a few tokens: h' = h + delta (h without one) and y [T, D] in
        the layer's type, the next block's delta.  Both are buffers of this
        block, which its next call overwrites."""
        d = self.decoder
        r = self.norm.forward(h, delta, stats=False)
        return h if r.h is None else r.h, d.decode(r.z)


class Q4Block:
    """The block around a layer of 4-bit expert weights: prompts by ``forward``, a few
    tokens by ``decode``, (h', y) from both as from a MoEBlock."""

    def __init__(self, norm: LayerNorm, layer: Q4Layer):
        if norm.D != layer.D:
            raise ValueError(f"the norm has {norm.D} channels, the layer {layer.D}")
        if norm.z_type != torch.bfloat16:
            raise ValueError(f"the norm writes {norm.z_type}, the layer reads bfloat16")
        if norm.device != layer.device:
            raise ValueError(f"the norm is on {norm.device}, the layer on {layer.device}")
        self.norm, self.layer = norm, layer

    def forward(self, h, delta=None):
        """h' = h + delta (h without one) and y [T, D] fp32, for up to the layer's
        max_tokens rows.  h' of up to 64 rows is a buffer of this block, which its next
        call overwrites."""
        r = self.norm.forward(h, delta, stats=False)
        return h if r.h is None else r.h, self.layer.forward(r.z)

    def decode(self, h, delta=None):
        """The same for a few tokens; y is in bf16.  Both are buffers of this block,
        which its next call overwrites."""
        r = self.norm.forward(h, delta, stats=False)
        return h if r.h is None else r.h, self.layer.decode(r.z)

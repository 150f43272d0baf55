"""The MoE layer on 4-bit expert weights, for serving, on top of the ctypes binding.

``Q4Layer`` holds references to the router's weights and the 4-bit expert matrices,
owns the workspace and calls ``moe_q4_forward`` (``include/moe_q4.h``); ``decoder`` is
its form for a few tokens, where it has one.  It computes nothing itself.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as B
from .decode import MoEDecoder, check_weights
from .layer import MoELayer
from .q4 import quantize

_MATRICES = ("w1", "w3", "w2", "ws1", "ws3", "ws2")


class Q4Layer:
    """w_gate [E,D] fp32; w1, w3 [E,F,D] and w2 [E,D,F] Q4Matrix; the shared branch ws1,
    ws3 [1,n_shared F,D] and ws2 [1,D,n_shared F] Q4Matrix; b1 [E,F], b2 [E,D], logit_bias
    [E], corr_bias [E] fp32 or None: used in place, in the storage that they have when the
    layer is made.  ``decoder`` is None where D, F or n_shared F are past the few-token
    form's limits (moe_decode's).  Calls run on the current stream of their GPU, which has
    to be the current one; those of one layer share its workspace and must not overlap on
    the GPU."""

    # calls pass addresses and configurations made from these once
    _FIXED = frozenset(("workspace", "cfg", "device", "D", "max_tokens", "matrices"))

    def __setattr__(self, name, value):
        if name in self._FIXED and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} is fixed when the layer is made")
        self.__dict__[name] = value

    def __init__(self, w_gate, w1, w2, w3=None, b1=None, b2=None, k=1, act="relu",
                 score="softmax", n_groups=1, topk_groups=1, group_score="top2_sum",
                 logit_bias=None, corr_bias=None, n_shared=0, ws1=None, ws3=None, ws2=None,
                 capacity_factor=0.0, max_tokens=4096):
        if max_tokens < 1:
            raise ValueError("max_tokens must be positive")
        args = dict(
            w3=w3, b1=b1, b2=b2, k=k, act=act, score=score, n_groups=n_groups,
            topk_groups=topk_groups, group_score=group_score, logit_bias=logit_bias,
            corr_bias=corr_bias, n_shared=n_shared, ws1=ws1, ws3=ws3, ws2=ws2,
            capacity_factor=capacity_factor)
        w = check_weights(w_gate, w1, w2, **args)
        if w.entry != "moe_q4_decode":
            raise ValueError("the expert weights must be Q4Matrix objects")
        if w.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
            raise ValueError("a layer cannot be made while its stream is being captured")
        self.device, self.D, self.max_tokens = w.device, w.D, int(max_tokens)
        self.matrices = {n: m for n, m in zip(_MATRICES, (w1, w3, w2, ws1, ws3, ws2)) if m is not None}
        self._make, self._hold, self._weights = w.make, w.hold, w.struct
        self._weights_ref = ctypes.byref(self._weights)
        self._calls = {}
        self.cfg = w.make(self.max_tokens)
        nbytes = B.moe_q4_workspace_size(self.cfg)
        if nbytes == 0:
            raise B.MoEError("moe_q4_workspace_size", B.MOE_ERR_INVALID_ARG,
                             "invalid or unsupported configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.workspace[:16].zero_()      # the status word, for a look before the first call
        few = min(self.max_tokens, B.MOE_DECODE_MAX_TOKENS)
        self.decoder: Optional[MoEDecoder] = None
        if B.moe_decode_workspace_size(w.make(few)) > 0:
            self.decoder = MoEDecoder(w_gate, w1, w2, max_tokens=few, **args)

    @classmethod
    def from_layer(cls, layer: MoELayer, group=64, max_tokens=None) -> "Q4Layer":
        """The 4-bit form of a bf16 layer: its expert weights (the fp32 masters) quantised,
        the router's and the biases used in place.  ``requantize`` follows further
        training."""
        if layer.dtype != "bf16":
            raise ValueError("only bf16 layers have a 4-bit form")
        c = layer.cfg
        name_of = lambda table, v: next(k for k, i in table.items() if i == v)  # noqa: E731
        masters = {n: getattr(layer, n) for n in _MATRICES}
        return cls(layer.w_gate, b1=layer.b1, b2=layer.b2, k=c.k, act=name_of(B.ACT, c.act),
                   score=name_of(B.SCORE, c.score), n_groups=c.n_groups, topk_groups=c.topk_groups,
                   group_score=name_of(B.GROUP_SCORE, c.group_score), logit_bias=layer.logit_bias,
                   corr_bias=layer.corr_bias, n_shared=c.n_shared,
                   capacity_factor=c.capacity_factor, max_tokens=max_tokens or max(c.T, 1),
                   **{n: None if w is None else quantize(w, group) for n, w in masters.items()})

    def requantize(self, layer: MoELayer):
        """Rewrites the 4-bit matrices from the layer's fp32 masters (of the shapes that
        this layer was made of)."""
        for n, m in self.matrices.items():
            quantize(getattr(layer, n), m.group, out=m)

    def forward(self, x, y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [T, D] fp32 of the tokens x [T, D] bf16, 0 <= T <= max_tokens."""
        shape = x.shape
        if (len(shape) != 2 or shape[1] != self.D or x.dtype is not torch.bfloat16 or
                x.device != self.device or not x.is_contiguous()):
            raise ValueError(f"x must be contiguous bfloat16 [T, {self.D}] on {self.device}, got "
                             f"{x.dtype} {tuple(shape)} on {x.device}")
        T = shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens: the layer was made for at most {self.max_tokens}")
        if y is None:
            y = torch.empty(T, self.D, dtype=torch.float32, device=self.device)
        elif (y.shape != shape or y.dtype is not torch.float32 or y.device != self.device or
              not y.is_contiguous()):
            raise ValueError(f"y must be contiguous float32 {tuple(shape)} on {self.device}")
        c = self._calls.get(T)
        if c is None:
            if len(self._calls) >= 64:
                self._calls.clear()
            cfg = self._make(T)
            c = self._calls[T] = cfg, ctypes.byref(cfg)
        status = B.lib().moe_q4_forward(c[1], self._weights_ref, x.data_ptr(), y.data_ptr(),
                                        self.workspace.data_ptr(), self.workspace.numel(),
                                        B._stream_on(None, self.device))
        if status != B.MOE_OK:
            B._check("moe_q4_forward", status)
        return y

    def decode(self, x, y=None):
        """y [T, D] bf16 for a few tokens (``MoEDecoder.decode``)."""
        if self.decoder is None:
            raise ValueError("D, F or n_shared F are past the few-token form's limits: use forward")
        return self.decoder.decode(x, y)

    def status(self) -> int:
        """Device status of the last ``forward`` of a token or more (0, or a MOE_ERR_* code).
        Waits for the current stream."""
        return B.moe_q4_status(self.cfg, self.workspace, B._stream_on(None, self.device))

"""The MoE layer for a few tokens (serving), on top of the ctypes binding.

``MoEDecoder`` holds references to one layer's weights, the workspace and the
output buffers, and calls ``moe_decode`` (``include/moe_block.h``).  It computes
nothing itself.
"""

from __future__ import annotations

import ctypes
from typing import Callable, NamedTuple

import torch

from . import binding as B
from .q4 import Q4Matrix

_DTYPE = {torch.float32: "f32", torch.bfloat16: "bf16"}


class Weights(NamedTuple):
    """The checked weights of a layer that serves, as the C ABI takes them."""
    device: torch.device
    dtype: torch.dtype        # the tokens' type
    D: int
    make: Callable            # the configuration for a number of tokens
    hold: list                # keeps the storage alive, even if a parameter's is replaced
    entry: str                # the few-token form's entry point
    struct: ctypes.Structure


def check_weights(w_gate, w1, w2, w3=None, b1=None, b2=None, k=1, act="relu", score="softmax",
                  n_groups=1, topk_groups=1, group_score="top2_sum", logit_bias=None,
                  corr_bias=None, n_shared=0, ws1=None, ws3=None, ws2=None,
                  capacity_factor=0.0) -> Weights:
    """The weights of a ``MoEDecoder`` (which describes them) or raises."""
    q4 = isinstance(w1, Q4Matrix)
    if not q4 and w1.dtype not in _DTYPE:
        raise ValueError(f"w1 must be float32, bfloat16 or a Q4Matrix, got {w1.dtype}")
    if len(w1.shape) != 3:
        raise ValueError(f"w1 must be [E, F, D], got {tuple(w1.shape)}")
    E, F, D = w1.shape
    Fs = int(n_shared) * F
    if (w3 is not None) != (act == "swiglu"):
        raise ValueError("w3 goes with swiglu experts, and only with them")
    if (b1 is None) != (b2 is None):
        raise ValueError("b1 and b2 come together")
    f32, dt = torch.float32, torch.bfloat16 if q4 else w1.dtype
    one = (1,) if q4 else ()
    want = dict(w_gate=(w_gate, f32, (E, D)), w1=(w1, dt, (E, F, D)), w2=(w2, dt, (E, D, F)),
                w3=(w3, dt, (E, F, D)), b1=(b1, f32, (E, F)), b2=(b2, f32, (E, D)),
                logit_bias=(logit_bias, f32, (E,)), corr_bias=(corr_bias, f32, (E,)),
                ws1=(ws1, dt, one + (Fs, D)), ws3=(ws3, dt, one + (Fs, D)),
                ws2=(ws2, dt, one + (D, Fs)))
    matrices = {}
    for name, (t, dtype, shape) in want.items():
        if name.startswith("ws") and (t is not None) != (n_shared > 0):
            raise ValueError("ws1, ws3 and ws2 go with n_shared > 0")
        if t is None:
            continue
        if q4 and dtype is dt:
            if not isinstance(t, Q4Matrix) or t.shape != shape or t.group != w1.group:
                raise ValueError(f"{name} must be a Q4Matrix of shape {shape} with groups of "
                                 f"{w1.group}, like w1")
            matrices[name] = t
        elif (isinstance(t, Q4Matrix) or t.dtype != dtype or tuple(t.shape) != shape or
              not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous {dtype} of shape {shape}, got "
                             f"{getattr(t, 'dtype', 'a Q4Matrix')} {tuple(t.shape)}")
        if t.device != w1.device:
            raise ValueError(f"{name} is on {t.device}, w1 on {w1.device}")

    def make(T):
        return B.make_config(T, D, F, E, k, act=act, score=score, n_groups=n_groups,
                             topk_groups=topk_groups, group_score=group_score, dtype=_DTYPE[dt],
                             has_bias=b1 is not None, n_shared=n_shared,
                             capacity_factor=capacity_factor)

    hold = [t._held if isinstance(t, Q4Matrix) else t.detach() for t, _, _ in want.values()
            if t is not None]
    if q4:
        entry = "moe_q4_decode"
        struct = B.make_q4_weights(w_gate, w1.group, b1=b1, b2=b2, logit_bias=logit_bias,
                                   corr_bias=corr_bias,
                                   **{n: m.c_matrix() for n, m in matrices.items()})
    else:
        entry = "moe_decode"
        struct = B.make_weights(w_gate, w1, w2, w3, b1, b2, logit_bias, corr_bias, ws1, ws3, ws2)
    return Weights(w1.device, dt, D, make, hold, entry, struct)


class MoEDecoder:
    """w_gate [E,D] fp32; w1, w3 [E,F,D], w2 [E,D,F] and the shared branch ws1,
    ws3, ws2 in the layer's type (float32 or bfloat16); b1 [E,F], b2 [E,D],
    logit_bias [E], corr_bias [E] fp32 or None.  Or all of w1, w3, w2, ws1, ws3, ws2 as
    Q4Matrix ([1, n_shared F, D] and [1, D, n_shared F] for the shared branch), of one
    group, in a bfloat16 layer (``moe_q4_decode``).  The tensors are used in place (in
    the storage that they have when the decoder is made), so the decoder follows
    a layer that is still being trained.  Calls run on the current stream of
    their GPU, which has to be the current one; those of one decoder share its
    buffers and must not overlap on the GPU, nor with the decoder's making, which
    clears its workspace on the current stream (and so cannot be part of a graph
    capture: the workspace would be cleared by the graph's replays only)."""

    # calls pass addresses and configurations made from these once
    _FIXED = frozenset(("workspace", "cfg", "device", "dtype", "D", "k", "max_tokens"))

    def __setattr__(self, name, value):
        if name in self._FIXED and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} is fixed when the decoder is made")
        self.__dict__[name] = value

    def __init__(self, w_gate, w1, w2, w3=None, b1=None, b2=None, k=1, act="relu",
                 score="softmax", n_groups=1, topk_groups=1, group_score="top2_sum",
                 logit_bias=None, corr_bias=None, n_shared=0, ws1=None, ws3=None, ws2=None,
                 capacity_factor=0.0, max_tokens=B.MOE_DECODE_MAX_TOKENS):
        if not 1 <= max_tokens <= B.MOE_DECODE_MAX_TOKENS:
            raise ValueError(f"max_tokens must be 1 to {B.MOE_DECODE_MAX_TOKENS}")
        w = check_weights(w_gate, w1, w2, w3, b1, b2, k, act, score, n_groups, topk_groups,
                          group_score, logit_bias, corr_bias, n_shared, ws1, ws3, ws2,
                          capacity_factor)
        if w.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
            raise ValueError("a decoder cannot be made while its stream is being captured")
        D, dt, f32 = w.D, w.dtype, torch.float32
        self.device, self.dtype, self.D, self.k = w.device, dt, D, int(k)
        self.max_tokens = int(max_tokens)
        self._make, self._hold, self._entry, self._weights = w.make, w.hold, w.entry, w.struct
        self._weights_ref = ctypes.byref(self._weights)
        self._calls = {}
        self.cfg = self._make(self.max_tokens)
        nbytes = B.moe_decode_workspace_size(self.cfg)
        if nbytes == 0:
            raise B.MoEError("moe_decode_workspace_size", B.MOE_ERR_INVALID_ARG,
                             "invalid or unsupported configuration")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._y = torch.empty(self.max_tokens, D, dtype=dt, device=self.device)
        self._idx = torch.empty(self.max_tokens, k, dtype=torch.int32, device=self.device)
        self._gate = torch.empty(self.max_tokens, k, dtype=f32, device=self.device)
        self.idx, self.gate = self._idx[:0], self._gate[:0]
        if self.device.type == "cuda":
            self.reset()     # on the current stream, which made the workspace as well

    def _call(self, T):
        """What a call on T tokens passes and hands out, made once per T."""
        cfg = self._make(T)
        c = self._calls[T] = (cfg, ctypes.byref(cfg), self._y[:T], self._idx[:T], self._gate[:T],
                              self._y.data_ptr(), self._idx.data_ptr(), self._gate.data_ptr(),
                              self.workspace.data_ptr(), self.workspace.numel())
        return c

    def decode(self, x, y=None):
        """y [T, D] of the tokens x [T, D] (the layer's type, 0 <= T <=
        max_tokens).  Without ``y`` the result is written to a buffer of the
        decoder, which the next call overwrites; ``idx`` and ``gate`` [T, k]
        hold the last call's routing, in buffers of the decoder as well."""
        shape = x.shape
        if (len(shape) != 2 or shape[1] != self.D or x.dtype != self.dtype or
                x.device != self.device or not x.is_contiguous()):
            raise ValueError(f"x must be contiguous {self.dtype} [T, {self.D}] on {self.device}, "
                             f"got {x.dtype} {tuple(shape)} on {x.device}")
        T = shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens: the decoder was made for at most {self.max_tokens}")
        c = self._calls.get(T) or self._call(T)
        if y is None:
            y, yp = c[2], c[5]
        else:
            if (y.shape != shape or y.dtype != self.dtype or y.device != self.device or
                    not y.is_contiguous()):
                raise ValueError(f"y must be contiguous {self.dtype} {tuple(shape)} on "
                                 f"{self.device}")
            yp = y.data_ptr()
        status = getattr(B.lib(), self._entry)(c[1], self._weights_ref, x.data_ptr(), yp, c[6],
                                               c[7], c[8], c[9], B._stream_on(None, self.device))
        if status != B.MOE_OK:
            B._check(self._entry, status)
        self.__dict__.update(idx=c[3], gate=c[4])      # (without __setattr__'s look-up)
        return y

    def status(self) -> int:
        """Device status since the last reset (0, or a MOE_ERR_* code; see
        moe_decode_status).  Waits for the current stream."""
        return B.moe_decode_status(self.cfg, self.workspace, B._stream_on(None, self.device))

    def reset(self):
        """Makes the workspace ready again after a status other than 0."""
        B.moe_decode_init(self.cfg, self.workspace, B._stream_on(None, self.device))

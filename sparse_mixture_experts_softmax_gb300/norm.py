"""Layer norm of a pre-norm residual block, on top of the ctypes binding.

``LayerNorm`` holds references to the fp32 parameters and the backward pass's
workspace, allocates outputs through torch and calls the C ABI of
``include/moe_block.h``.  It computes nothing itself.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import binding as B

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
_TYPE = {torch.float32: B.DTYPE["f32"], torch.bfloat16: B.DTYPE["bf16"]}


class NormOut(NamedTuple):
    h: Optional[torch.Tensor]      # the updated stream, or None without a delta
    z: torch.Tensor
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


class NormGrads(NamedTuple):
    dx: torch.Tensor
    dgamma: torch.Tensor
    dbeta: Optional[torch.Tensor]


class LayerNorm:
    """gamma, beta (or None): fp32 [D] on the GPU, used in place (the storage that
    they have when the object is made); they change in place only.  x_dtype is the
    residual stream's type, z_dtype the following layer's input type.  Calls run on
    the current stream of their GPU, which has to be the current one; those of one
    object share its buffers, so they must not overlap on the GPU (several streams:
    order them, or give ``out`` and use an object each)."""

    # calls pass addresses and configurations made from these once
    _FIXED = frozenset(("gamma", "beta", "D", "device", "x_type", "z_type", "eps"))

    def __setattr__(self, name, value):
        if name in self._FIXED and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} is fixed when the norm is made (gamma and beta change "
                                 "in place)")
        self.__dict__[name] = value

    def __init__(self, gamma, beta=None, x_dtype="f32", z_dtype="f32", eps=1e-5):
        self.D = int(gamma.numel())
        for name, p in (("gamma", gamma), ("beta", beta)):
            if p is not None and (p.dtype != torch.float32 or tuple(p.shape) != (self.D,) or
                                  not p.is_contiguous()):
                raise ValueError(f"{name} must be contiguous float32 of shape [{self.D}]")
        if beta is not None and beta.device != gamma.device:
            raise ValueError(f"beta is on {beta.device}, gamma on {gamma.device}")
        # (detached: they keep that storage even if a parameter's is replaced)
        self.gamma, self.beta = gamma.detach(), None if beta is None else beta.detach()
        # what the addresses below are of, whatever becomes of the attributes' storage
        self._held = gamma.detach(), None if beta is None else beta.detach()
        self._gamma_ptr = gamma.data_ptr()
        self._beta_ptr = None if beta is None else beta.data_ptr()
        self.device = gamma.device
        self.x_type, self.z_type, self.eps = _TORCH[x_dtype], _TORCH[z_dtype], float(eps)
        self.workspace = self.dgamma = self.dbeta = None
        self._plans, self._own = {}, {}

    def _plan(self, shape, delta):
        """What a call on rows of `shape` passes besides its tensors: the C
        configuration, its reference, and a tensor like its statistics.  The last ones are kept: a program passes
        the same shapes over and over, and a call costs as much host time as a
        small kernel runs."""
        if len(shape) != 2 or shape[1] != self.D:
            raise ValueError(f"the rows must be [T, {self.D}], got {tuple(shape)}")
        if delta is not None and delta not in _TYPE:
            raise ValueError(f"delta must be float32 or bfloat16, got {delta}")
        if len(self._plans) >= 64:
            self._plans.clear()
        cfg = B.moe_norm_config(shape[0], self.D, _TYPE[self.x_type], _TYPE[delta or torch.float32],
                                _TYPE[self.z_type], self.eps)
        p = self._plans[shape, delta] = (
            cfg, ctypes.byref(cfg),
            torch.empty(shape[0], dtype=torch.float32, device=self.device))
        return p

    def _buffers(self, shape, plain):
        """Outputs of a call without statistics.  Those of few rows stay for
        good: a captured graph writes to them as long as it lives."""
        new = lambda dtype: torch.empty(shape, dtype=dtype, device=self.device)  # noqa: E731
        out = NormOut(None if plain else new(self.x_type), new(self.z_type), None, None)
        if shape[0] <= B.MOE_DECODE_MAX_TOKENS:
            self._own[shape, plain] = out
        return out

    def _wrong(self, name, t, dtype, shape):
        """Raises for a tensor that is not contiguous `dtype` of `shape` on the
        parameters' device."""
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the parameters on {self.device}")
        raise ValueError(f"{name} must be contiguous {dtype} of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")

    def _rows(self, name, t, dtype, shape):
        if (t.dtype is not dtype or t.shape != shape or t.device != self.device or
                not t.is_contiguous()):
            self._wrong(name, t, dtype, shape)

    def forward(self, x, delta=None, stats=True, out=None) -> NormOut:
        """h = x + delta (x itself without a delta), z = norm(h).  ``out``: a
        NormOut whose tensors are written instead of new ones; its h may be
        ``x``.  stats=False (serving) leaves mean and rstd out, and without
        ``out`` writes h and z of up to 64 rows to buffers of this object, which
        its next such call overwrites: allocating two tensors takes as long as
        launching the kernel does."""
        shape = x.shape
        kind = None if delta is None else delta.dtype
        plan = self._plans.get((shape, kind)) or self._plan(shape, kind)
        if x.dtype is not self.x_type or x.device != self.device or not x.is_contiguous():
            self._wrong("x", x, self.x_type, shape)
        if delta is not None and (delta.shape != shape or delta.device != self.device or
                                  not delta.is_contiguous()):
            self._wrong("delta", delta, kind, shape)
        if out is not None:
            T = shape[0]
            if (out.h is not None) != (delta is not None):
                raise ValueError("out.h goes with a delta")
            if out.h is not None:
                self._rows("out.h", out.h, self.x_type, shape)
            self._rows("out.z", out.z, self.z_type, shape)
            for name, t in (("out.mean", out.mean), ("out.rstd", out.rstd)):
                if t is not None:
                    self._rows(name, t, torch.float32, (T,))
        elif stats:
            like = torch.empty_like
            out = NormOut(None if delta is None else like(x),
                          like(x) if self.z_type is self.x_type else like(x, dtype=self.z_type),
                          like(plan[2]), like(plan[2]))
        else:
            out = self._own.get((shape, delta is None)) or self._buffers(shape, delta is None)
        h, z, mean, rstd = out
        status = B.lib().moe_norm_forward(
            plan[1], x.data_ptr(), None if delta is None else delta.data_ptr(), self._gamma_ptr,
            self._beta_ptr, None if h is None else h.data_ptr(), z.data_ptr(),
            None if mean is None else mean.data_ptr(), None if rstd is None else rstd.data_ptr(),
            B._stream_on(None, self.device))
        if status != B.MOE_OK:
            B._check("moe_norm_forward", status)
        return out

    def backward(self, dz, h, mean, rstd, dres=None, out=None) -> NormGrads:
        """Gradients at the stream h that ``forward`` normalised (its h, or its
        x without a delta); dres: the gradient reaching h past the norm.
        ``out``: a NormGrads to write; its dx may be ``dz`` or ``dres``.  Without
        it dx is new, and the parameters' gradients are written to ``dgamma``
        and ``dbeta`` of this object (overwritten, never added to, as a layer's
        own gradient buffers are)."""
        shape = h.shape
        plan = self._plans.get((shape, None)) or self._plan(shape, None)
        T, f32 = shape[0], torch.float32
        self._rows("h", h, self.x_type, shape)
        self._rows("dz", dz, f32, shape)
        self._rows("mean", mean, f32, (T,))
        self._rows("rstd", rstd, f32, (T,))
        if dres is not None:
            self._rows("dres", dres, f32, shape)
        if out is None:
            if self.dgamma is None:
                self.dgamma = torch.empty_like(self.gamma)
                self.dbeta = None if self.beta is None else torch.empty_like(self.beta)
            out = NormGrads(torch.empty_like(dz), self.dgamma, self.dbeta)
        else:
            self._rows("out.dx", out.dx, f32, shape)
            self._rows("out.dgamma", out.dgamma, f32, (self.D,))
            if out.dbeta is not None:
                self._rows("out.dbeta", out.dbeta, f32, (self.D,))
        if self.workspace is None:
            # for any number of rows, so that it is never replaced under a graph that uses it
            most = B.moe_norm_workspace_size(B.make_norm_config(2**31 - 1, self.D))
            self.workspace = torch.empty(most, dtype=torch.uint8, device=self.device)
        status = B.lib().moe_norm_backward(
            plan[1], h.data_ptr(), dz.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            self._gamma_ptr, None if dres is None else dres.data_ptr(), out.dx.data_ptr(),
            out.dgamma.data_ptr(), None if out.dbeta is None else out.dbeta.data_ptr(),
            self.workspace.data_ptr(), self.workspace.numel(), B._stream_on(None, self.device))
        if status != B.MOE_OK:
            B._check("moe_norm_backward", status)
        return out

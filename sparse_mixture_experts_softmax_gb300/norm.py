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
    """gamma, beta (or None): fp32 [D] on the GPU, used in place.  x_dtype is
    the residual stream's type, z_dtype the following layer's input type."""

    def __init__(self, gamma, beta=None, x_dtype="f32", z_dtype="f32", eps=1e-5):
        self.D = int(gamma.numel())
        for name, p in (("gamma", gamma), ("beta", beta)):
            if p is not None and (p.dtype != torch.float32 or tuple(p.shape) != (self.D,)):
                raise ValueError(f"{name} must be float32 of shape [{self.D}]")
        if beta is not None and beta.device != gamma.device:
            raise ValueError(f"beta is on {beta.device}, gamma on {gamma.device}")
        self.gamma, self.beta, self.device = gamma, beta, gamma.device
        self.x_type, self.z_type, self.eps = _TORCH[x_dtype], _TORCH[z_dtype], float(eps)
        self.workspace = self.dgamma = self.dbeta = None
        self._cfg, self._own = {}, {}

    def _config(self, T, delta):
        """The C configuration of T rows, its reference, and the backward
        pass's workspace size (the last configurations are kept: a decoding
        program passes the same T over and over)."""
        key = (T, delta)
        c = self._cfg.get(key)
        if c is None:
            if len(self._cfg) >= 256:
                self._cfg.clear()
            cfg = B.moe_norm_config(T, self.D, _TYPE[self.x_type], _TYPE[delta],
                                    _TYPE[self.z_type], self.eps)
            c = self._cfg[key] = (cfg, ctypes.byref(cfg), B.moe_norm_workspace_size(cfg))
        return c

    def _buffers(self, T, plain):
        """Outputs of a call without statistics; one size at a time is kept."""
        self._own.clear()
        new = lambda dtype: torch.empty(T, self.D, dtype=dtype, device=self.device)  # noqa: E731
        out = self._own[T, plain] = NormOut(None if plain else new(self.x_type), new(self.z_type),
                                            None, None)
        return out

    def _wrong(self, name, t, dtype, shape):
        """Raises for a tensor that is not contiguous `dtype` of `shape` on the
        parameters' device."""
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the parameters on {self.device}")
        raise ValueError(f"{name} must be contiguous {dtype} of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")

    def _rows(self, name, t, dtype, shape):
        if (t.dtype != dtype or t.shape != shape or t.device != self.device or
                not t.is_contiguous()):
            self._wrong(name, t, dtype, shape)

    def forward(self, x, delta=None, stats=True, out=None, stream=None) -> NormOut:
        """h = x + delta (x itself without a delta), z = norm(h).  ``out``: a
        NormOut whose tensors are written instead of new ones; its h may be
        ``x``.  stats=False (serving) leaves mean and rstd out, and without
        ``out`` writes h and z to buffers of this object, which its next such
        call overwrites: allocating two tensors takes as long as launching the
        kernel does."""
        shape = x.shape
        if len(shape) != 2 or shape[1] != self.D:
            raise ValueError(f"x must be [T, {self.D}], got {tuple(shape)}")
        T = shape[0]
        self._rows("x", x, self.x_type, shape)
        if delta is not None:
            if delta.dtype not in _TYPE:
                raise ValueError(f"delta must be float32 or bfloat16, got {delta.dtype}")
            self._rows("delta", delta, delta.dtype, shape)
        if out is None:
            if stats:
                out = NormOut(torch.empty_like(x) if delta is not None else None,
                              torch.empty_like(x, dtype=self.z_type),
                              torch.empty(T, dtype=torch.float32, device=self.device),
                              torch.empty(T, dtype=torch.float32, device=self.device))
            else:
                out = self._own.get((T, delta is None)) or self._buffers(T, delta is None)
        else:
            if (out.h is not None) != (delta is not None):
                raise ValueError("out.h goes with a delta")
            if out.h is not None:
                self._rows("out.h", out.h, self.x_type, shape)
            self._rows("out.z", out.z, self.z_type, shape)
            for name, t in (("out.mean", out.mean), ("out.rstd", out.rstd)):
                if t is not None:
                    self._rows(name, t, torch.float32, (T,))
        cfg = self._config(T, delta.dtype if delta is not None else torch.float32)
        B._check("moe_norm_forward", B.lib().moe_norm_forward(
            cfg[1], x.data_ptr(), None if delta is None else delta.data_ptr(),
            self.gamma.data_ptr(), B._ptr(self.beta), None if delta is None else out.h.data_ptr(),
            out.z.data_ptr(), B._ptr(out.mean), B._ptr(out.rstd), B._stream_on(stream, self.device)))
        return out

    def backward(self, dz, h, mean, rstd, dres=None, out=None, stream=None) -> NormGrads:
        """Gradients at the stream h that ``forward`` normalised (its h, or its
        x without a delta); dres: the gradient reaching h past the norm.
        ``out``: a NormGrads to write; its dx may be ``dz`` or ``dres``.  Without
        it dx is new, and the parameters' gradients are written to ``dgamma``
        and ``dbeta`` of this object (overwritten, never added to, as a layer's
        own gradient buffers are)."""
        shape = h.shape
        if len(shape) != 2 or shape[1] != self.D:
            raise ValueError(f"h must be [T, {self.D}], got {tuple(shape)}")
        T = shape[0]
        self._rows("h", h, self.x_type, shape)
        self._rows("dz", dz, torch.float32, shape)
        self._rows("mean", mean, torch.float32, (T,))
        self._rows("rstd", rstd, torch.float32, (T,))
        if dres is not None:
            self._rows("dres", dres, torch.float32, shape)
        if out is None:
            if self.dgamma is None:
                self.dgamma = torch.empty_like(self.gamma)
                self.dbeta = None if self.beta is None else torch.empty_like(self.beta)
            out = NormGrads(torch.empty_like(dz), self.dgamma, self.dbeta)
        else:
            self._rows("out.dx", out.dx, torch.float32, shape)
            self._rows("out.dgamma", out.dgamma, torch.float32, (self.D,))
            if out.dbeta is not None:
                self._rows("out.dbeta", out.dbeta, torch.float32, (self.D,))
        cfg = self._config(T, torch.float32)
        if self.workspace is None or self.workspace.numel() < cfg[2]:
            self.workspace = torch.empty(cfg[2], dtype=torch.uint8, device=h.device)
        B._check("moe_norm_backward", B.lib().moe_norm_backward(
            cfg[1], h.data_ptr(), dz.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            self.gamma.data_ptr(), B._ptr(dres), out.dx.data_ptr(), out.dgamma.data_ptr(),
            B._ptr(out.dbeta), self.workspace.data_ptr(), self.workspace.numel(),
            B._stream_on(stream, self.device)))
        return out

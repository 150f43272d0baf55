"""4-bit expert weights, on top of the ctypes binding (``include/moe_q4.h``).

``quantize`` makes a ``Q4Matrix`` of an expert matrix; ``Q4Product`` multiplies the
rows of each expert with one.  Nothing is computed here: outputs are allocated
through torch and the C ABI is called, on the current stream of the tensors' GPU,
which has to be the current one.
"""

from __future__ import annotations

import ctypes

import torch

from . import binding as B

_CODE = {torch.float32: B.DTYPE["f32"], torch.bfloat16: B.DTYPE["bf16"]}


def _want(name, t, dtype, shape, device):
    """Raises unless t is contiguous `dtype` of `shape` on `device`."""
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


class Q4Matrix:
    """A 4-bit matrix [E, N, K] (N outputs, K inputs of each of E experts):

    codes   uint8 [E, N, K / 2], 32-bit words of eight inputs each, input i of a word's
            eight in its four bits from 4 (i // 2) + 16 (i % 2) on;
    scales  bfloat16 [E, ceil(K / group), N];

    it stands for the weights (code - 8) scale, rounded to bfloat16.  The tensors are
    used in place (in the storage that they have when the object is made) and change in
    place only."""

    __slots__ = ("_codes", "_scales", "_group", "_shape", "_device", "_held", "_c", "_ref")

    def __init__(self, codes, scales, group):
        if group not in B.Q4_GROUPS:
            raise ValueError(f"group must be one of {B.Q4_GROUPS}, got {group}")
        if codes.dim() != 3:
            raise ValueError(f"codes must be [E, N, K / 2], got {tuple(codes.shape)}")
        E, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
        if E < 1 or N < 1 or K < 1 or N % 8 or K % 32:
            raise ValueError(f"N must be a multiple of 8 and K of 32, got {(E, N, K)}")
        _want("codes", codes, torch.uint8, (E, N, K // 2), codes.device)
        _want("scales", scales, torch.bfloat16, (E, -(-K // group), N), codes.device)
        self._set(codes.detach(), scales.detach(), int(group), (E, N, K))

    def _set(self, codes, scales, group, shape):
        self._codes, self._scales, self._group, self._shape = codes, scales, group, shape
        self._device = codes.device
        # what the addresses are of, whatever becomes of the attributes' storage
        self._held = codes.detach(), scales.detach()
        self._c = c = B.moe_q4_matrix(codes.data_ptr(), scales.data_ptr())
        self._ref = ctypes.byref(c)

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    group = property(lambda self: self._group)
    shape = property(lambda self: self._shape)
    device = property(lambda self: self._device)
    E = property(lambda self: self._shape[0])
    N = property(lambda self: self._shape[1])
    K = property(lambda self: self._shape[2])

    def c_matrix(self) -> B.moe_q4_matrix:
        """The matrix as the C ABI takes it; it keeps no tensor alive."""
        return B.moe_q4_matrix(self._c.codes, self._c.scales)

    def dequantize(self, dtype=torch.bfloat16, out=None):
        """The weights [E, N, K] (bfloat16 values, in float32 where asked)."""
        kind = _CODE.get(dtype if out is None else out.dtype)
        if kind is None:
            raise ValueError("the weights are float32 or bfloat16, not "
                             f"{dtype if out is None else out.dtype}")
        if out is None:
            out = torch.empty(self._shape, dtype=dtype, device=self._device)
        else:
            _want("out", out, out.dtype, self._shape, self._device)
        E, N, K = self._shape
        status = B.lib().moe_q4_dequantize(E, N, K, self._group, kind, self._ref, out.data_ptr(),
                                           B._stream_on(None, self._device))
        if status != B.MOE_OK:
            B._check("moe_q4_dequantize", status)
        return out


def quantize(w, group=64, out=None) -> Q4Matrix:
    """The 4-bit matrix of w [E, N, K] or [N, K] (then E is 1), float32 or bfloat16.  A
    group's scale is the smallest value of five significant bits that is not below
    max |w| / 7 (the smallest multiple of 2^-130 where that is below 2^-126), its codes
    8 + the nearest whole numbers to w / scale.  ``out``: a matrix of that shape and group
    that is rewritten (what was made with it follows)."""
    kind, device = _CODE.get(w.dtype), w.device
    if kind is None:
        raise ValueError(f"w must be float32 or bfloat16, got {w.dtype}")
    if group not in B.Q4_GROUPS:
        raise ValueError(f"group must be one of {B.Q4_GROUPS}, got {group}")
    shape = (1,) * (w.dim() == 2) + tuple(w.shape)
    if len(shape) != 3 or 0 in shape or shape[1] % 8 or shape[2] % 32 or not w.is_contiguous():
        raise ValueError("w must be contiguous [E, N, K] with N a multiple of 8 and K of 32, got "
                         f"{tuple(w.shape)}")
    E, N, K = shape
    if out is None:
        out = Q4Matrix.__new__(Q4Matrix)
        out._set(torch.empty((E, N, K // 2), dtype=torch.uint8, device=device),
                 torch.empty((E, -(-K // group), N), dtype=torch.bfloat16, device=device), group, shape)
    elif out.shape != shape or out.group != group or out.device != device:
        raise ValueError(f"out is {out.shape} with groups of {out.group} on {out.device}, w asks "
                         f"for {shape} with groups of {group} on {device}")
    status = B.lib().moe_q4_quantize(E, N, K, group, kind, w.data_ptr(), out._c.codes, out._c.scales,
                                     B._stream_on(None, device))
    if status != B.MOE_OK:
        B._check("moe_q4_quantize", status)
    return out


class Q4Product:
    """c[r] = act(W_e x[r] + bias_e) for the rows r of each expert e, or with act
    "swiglu"  SiLU(W_e x[r]) * (W3_e x[r]):  w (and w3) are Q4Matrix [E, N, K], bias is
    float32 [E, N] or None, act "none", "relu", "gelu_tanh" or "swiglu".  The tensors are
    used in place, in the storage that they have when the object is made.  Calls of one
    object share nothing but the status word, so they may overlap on the GPU; the first
    one has to come after the object's making, which clears that word on the current
    stream (and so cannot be part of a graph capture)."""

    _FIXED = frozenset(("shape", "device", "dev_status"))

    def __setattr__(self, name, value):
        if name in self._FIXED and name in self.__dict__:
            raise AttributeError(f"{name} is fixed when the product is made")
        self.__dict__[name] = value

    def __init__(self, w, w3=None, bias=None, act="none"):
        if act not in B.Q4_ACT:
            raise ValueError(f"act must be one of {sorted(B.Q4_ACT)}, got {act!r}")
        if (w3 is not None) != (act == "swiglu"):
            raise ValueError("w3 goes with swiglu, and only with it")
        if w.E > B.MOE_Q4_MAX_EXPERTS:
            raise ValueError(f"{w.E} experts: at most {B.MOE_Q4_MAX_EXPERTS}")
        if w3 is not None and (w3.shape != w.shape or w3.group != w.group or w3.device != w.device):
            raise ValueError(f"w3 is {w3.shape} with groups of {w3.group} on {w3.device}, w "
                             f"{w.shape} with groups of {w.group} on {w.device}")
        if bias is not None:
            if w3 is not None:
                raise ValueError("a swiglu product has no bias")
            _want("bias", bias, torch.float32, (w.E, w.N), w.device)
        if w.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
            raise ValueError("a product cannot be made while its stream is being captured")
        self.shape, self.device = w.shape, w.device
        self._offsets_shape = torch.Size((w.E + 1,))
        self._held = w._held, None if w3 is None else w3._held, None if bias is None else bias.detach()
        self._w = w.c_matrix()
        self._w3 = None if w3 is None else w3.c_matrix()
        self._refs = ctypes.byref(self._w), None if w3 is None else ctypes.byref(self._w3)
        self._bias = None if bias is None else bias.data_ptr()
        self._make = lambda R: B.moe_q4_product_config(R, w.E, w.N, w.K, w.group, B.Q4_ACT[act])  # noqa: E731
        self._calls = {}
        self.dev_status = torch.zeros(4, dtype=torch.int32, device=w.device)
        self._status = self.dev_status.data_ptr()

    def forward(self, x, offsets, out=None):
        """c [R, N] bfloat16 of the rows x [R, K] bfloat16.  The rows of expert e are
        offsets[e] to offsets[e + 1] - 1 (int32 [E + 1], on the GPU); values that decrease
        or leave 0 .. R are clamped.  Rows outside of every expert's reach no result and are
        left as they are in ``out`` (undefined without one), which must not overlap x."""
        E, N, K = self.shape
        device, shape = self.device, x.shape
        if (len(shape) != 2 or shape[1] != K or x.dtype is not torch.bfloat16 or
                x.device != device or not x.is_contiguous()):
            raise ValueError(f"x must be contiguous bfloat16 [R, {K}] on {device}, got {x.dtype} "
                             f"{tuple(shape)} on {x.device}")
        if (offsets.dtype is not torch.int32 or offsets.shape != self._offsets_shape or
                offsets.device != device or not offsets.is_contiguous()):
            raise ValueError(f"offsets must be contiguous int32 [{E + 1}] on {device}, got "
                             f"{offsets.dtype} {tuple(offsets.shape)} on {offsets.device}")
        R = shape[0]
        c = self._calls.get(R)
        if c is None:
            if len(self._calls) >= 64:
                self._calls.clear()
            cfg = self._make(R)
            # (a new tensor like another takes half the time of one from its shape; those kept
            # for it are of 512 KB at most)
            small = R <= 64 and R * N <= 1 << 18
            like = torch.empty((R, N), dtype=torch.bfloat16, device=device) if small else None
            c = self._calls[R] = cfg, ctypes.byref(cfg), like
        if out is not None:
            _want("out", out, torch.bfloat16, (R, N), device)
        elif c[2] is not None:
            out = torch.empty_like(c[2])
        else:
            out = torch.empty((R, N), dtype=torch.bfloat16, device=device)
        status = B.lib().moe_q4_product(c[1], offsets.data_ptr(), x.data_ptr(), self._refs[0],
                                        self._refs[1], self._bias, out.data_ptr(), self._status,
                                        B._stream_on(None, device))
        if status != B.MOE_OK:
            B._check("moe_q4_product", status)
        return out

    def status(self) -> int:
        """0, or MOE_ERR_TIMEOUT when a bounded device-side wait of a call expired (its
        output is invalid) since the object was made.  Waits for the current stream."""
        return int(self.dev_status[0])

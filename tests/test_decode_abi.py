"""Refusals and sizes of the few-token layer's entry points (host checks, no GPU)."""

import ctypes
import os

import pytest
import torch

from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.build import LIB, build_library
from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder

A = 0x7f0000000000          # a fake aligned address: host checks never follow it


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB):
        build_library()
    return B.lib()


def _cfg(**kw):
    base = dict(T=4, D=64, F=32, E=8, k=2, act="swiglu", score="softmax", dtype="bf16",
                has_bias=False)
    base.update(kw)
    return B.make_config(**base)


def _weights(**kw):
    w = B.moe_weights(*[A] * 11)
    for n, v in kw.items():
        setattr(w, n, v)
    return w


def _call(L, c, w=None, x=A, y=A, idx=A, gate=A, ws=A, nbytes=1 << 40):
    w = _weights() if w is None else w
    return L.moe_decode(ctypes.byref(c) if c is not None else None, ctypes.byref(w), x, y, idx,
                        gate, ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(T=65), dict(T=1 << 20), dict(D=(1 << 20) + 8),
                                dict(F=(1 << 19) + 8), dict(k=9), dict(D=60), dict(E=12),
                                dict(D=16392), dict(F=8200), dict(F=4104, n_shared=2),
                                dict(D=8200, act="relu", dtype="f32")])
def test_unsupported(L, kw):
    c = _cfg(**kw)
    assert B.moe_decode_workspace_size(c) == 0
    assert _call(L, c) == B.MOE_ERR_UNSUPPORTED
    assert L.moe_decode_init(ctypes.byref(c), A, 1 << 40, None) == B.MOE_ERR_UNSUPPORTED


def test_invalid(L):
    assert B.MOE_DECODE_MAX_TOKENS == 64
    c = _cfg()
    assert _call(L, None) == B.MOE_ERR_INVALID_ARG
    assert _call(L, _cfg(T=-1)) == B.MOE_ERR_INVALID_ARG
    assert L.moe_decode(ctypes.byref(c), None, A, A, A, A, A, 1 << 40, None) == \
        B.MOE_ERR_INVALID_ARG
    for n in ("w_gate", "w1", "w3", "w2"):
        assert _call(L, c, _weights(**{n: None})) == B.MOE_ERR_INVALID_ARG
    for n in ("ws1", "ws3", "ws2"):
        assert _call(L, _cfg(n_shared=1), _weights(**{n: None})) == B.MOE_ERR_INVALID_ARG
    biased = _cfg(act="relu", has_bias=True, dtype="f32")
    for n in ("b1", "b2"):
        assert _call(L, biased, _weights(**{n: None})) == B.MOE_ERR_INVALID_ARG
    assert _call(L, c, x=None) == B.MOE_ERR_INVALID_ARG
    assert _call(L, c, y=None) == B.MOE_ERR_INVALID_ARG
    assert _call(L, c, ws=None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_decode_init(ctypes.byref(c), None, 1 << 40, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_decode_status(ctypes.byref(c), A, 1 << 40, None, None) == B.MOE_ERR_INVALID_ARG


def test_alignment_and_workspace(L):
    c = _cfg()
    for n, _ in B.moe_weights._fields_:
        assert _call(L, c, _weights(**{n: A + 8})) == B.MOE_ERR_ALIGNMENT
    for n in ("x", "y", "idx", "gate", "ws"):
        assert _call(L, c, **{n: A + 4}) == B.MOE_ERR_ALIGNMENT
    need = B.moe_decode_workspace_size(c)
    assert need >= 4 * 8 * 4 + 4 * 2 * 32 * 4
    assert _call(L, c, nbytes=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
    assert L.moe_decode_init(ctypes.byref(c), A, need - 1, None) == B.MOE_ERR_WORKSPACE_TOO_SMALL


def test_workspace_grows_with_tokens(L):
    sizes = [B.moe_decode_workspace_size(_cfg(T=T, n_shared=1)) for T in range(65)]
    assert all(s > 0 for s in sizes) and sizes == sorted(sizes)


def test_python_refusals(L):
    E, F, D = 8, 16, 32
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    wg, w1, w2 = t(E, D, dt=torch.float32), t(E, F, D), t(E, D, F)
    ok = dict(k=2, act="relu")
    with pytest.raises(ValueError):
        MoEDecoder(wg.bfloat16(), w1, w2, **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1.half(), w2.half(), **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w2.float(), **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w1, **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1.transpose(1, 2), w2, **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w2, k=2, act="swiglu")              # no w3
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w2, w3=w1, **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w2, b1=t(E, F, dt=torch.float32), **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w2, n_shared=1, **ok)
    with pytest.raises(ValueError):
        MoEDecoder(wg, w1, w2, ws1=t(F, D), **ok)
    for m in (0, 65):
        with pytest.raises(ValueError):
            MoEDecoder(wg, w1, w2, max_tokens=m, **ok)
    with pytest.raises(B.MoEError):
        MoEDecoder(wg, w1, w2, k=9, act="relu")
    d = MoEDecoder(wg, w1, w2, max_tokens=4, **ok)
    for bad in (t(5, D), t(D), t(2, D + 1), t(2, D, dt=torch.float32), t(D, 2).t()):
        with pytest.raises(ValueError):
            d.decode(bad)
    with pytest.raises(ValueError):
        d.decode(t(2, D), y=t(3, D))
    with pytest.raises(ValueError):
        d.decode(t(2, D), y=t(2, D, dt=torch.float32))


def test_python_refuses_host_tensors(L):
    t = lambda *s: torch.zeros(*s)  # noqa: E731
    d = MoEDecoder(t(8, 32), t(8, 16, 32), t(8, 32, 16), k=2, max_tokens=4)
    with pytest.raises(ValueError, match="GPU"):
        d.decode(t(2, 32))


def test_what_a_decoder_is_made_of_stays(L):
    """Calls pass addresses taken once: a replaced workspace would be freed under them."""
    t = lambda *s: torch.zeros(*s)  # noqa: E731
    d = MoEDecoder(t(8, 32), t(8, 16, 32), t(8, 32, 16), k=2, max_tokens=4)
    for name in ("workspace", "cfg", "device", "dtype", "D", "k", "max_tokens"):
        with pytest.raises(AttributeError, match=name):
            setattr(d, name, None)

"""4-bit expert weights without a GPU: the packed layout's plain form, refusals of the
entry points (host checks) and of the Python classes, and the structs' layout."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.build import INCLUDE, LIB, build_library
from sparse_mixture_experts_softmax_gb300.q4 import Q4Matrix, Q4Product, quantize
from tests import q4_cases as C

A = 0x7f0000000000          # a fake aligned address: host checks never follow it


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB):
        build_library()
    return B.lib()


def test_layout_of_a_word():
    codes = np.arange(8).reshape(1, 1, 8)
    assert C.pack(codes).reshape(-1).tolist() == [0 | 2 << 4, 4 | 6 << 4, 1 | 3 << 4, 5 | 7 << 4]
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (2, 8, 96))
    assert np.array_equal(C.unpack(C.pack(codes)), codes)


@pytest.mark.parametrize("group", B.Q4_GROUPS)
def test_quantize_definition(group):
    w = np.random.default_rng(1).normal(0, 1, (2, 8, 160)).astype(np.float32).astype(np.float64)
    codes, scales = C.quantize(w, group)
    assert codes.min() >= 1 and codes.max() <= 15
    of = np.repeat(scales, group, axis=1)[:, :160].transpose(0, 2, 1)
    assert (np.abs(w - (codes - 8) * of) <= of / 2).all()
    assert np.array_equal((codes - 8) * of, C.weights(codes, scales, group))     # exact in bf16
    amax = np.stack([np.abs(w[..., g:g + group]).max(-1) for g in range(0, 160, group)], 1)
    assert (scales >= amax / 7).all() and (scales < amax / 7 * (1 + 2.0 ** -4)).all()


def _cfg(**kw):
    base = dict(R=4, E=3, N=16, K=64, group=32, act=B.MOE_Q4_ACT_NONE)
    base.update(kw)
    return B.moe_q4_product_config(*[base[n] for n, _ in B.moe_q4_product_config._fields_])


def _m(codes=A, scales=A):
    return ctypes.byref(B.moe_q4_matrix(codes, scales))


def _call(L, cfg, off=A, x=A, w=True, w3=None, bias=None, c=A, status=A):
    return L.moe_q4_product(None if cfg is None else ctypes.byref(cfg), off, x,
                            _m() if w is True else w, w3, bias, c, status, None)


@pytest.mark.parametrize("kw", [dict(N=12), dict(K=48), dict(group=16), dict(group=0), dict(group=48),
                                dict(E=257), dict(N=1 << 28, K=1 << 12), dict(E=256, N=1 << 23),
                                dict(R=2**31 - 1, K=1 << 12), dict(R=2**31 - 1, N=1 << 12),
                                dict(R=(1 << 30) + 1), dict(R=1, K=(1 << 28) + 32),
                                dict(E=1, N=(1 << 28) + 8)])
def test_product_unsupported(L, kw):
    assert _call(L, _cfg(**kw)) == B.MOE_ERR_UNSUPPORTED


def test_product_invalid(L):
    bad = B.MOE_ERR_INVALID_ARG
    assert _call(L, None) == bad
    for kw in (dict(R=-1), dict(E=0), dict(N=0), dict(K=0), dict(N=-8), dict(act=-1), dict(act=4)):
        assert _call(L, _cfg(**kw)) == bad
    for kw in (dict(off=None), dict(x=None), dict(w=None), dict(c=None), dict(status=None),
               dict(w=_m(codes=None)), dict(w=_m(scales=None)), dict(w3=_m())):
        assert _call(L, _cfg(), **kw) == bad
    swiglu = _cfg(act=B.ACT["swiglu"])
    assert _call(L, swiglu) == bad
    assert _call(L, swiglu, w3=_m(codes=None)) == bad
    assert _call(L, swiglu, w3=_m(), bias=A) == bad


def test_product_alignment(L):
    for kw in (dict(off=A + 4), dict(x=A + 8), dict(c=A + 2), dict(status=A + 4), dict(bias=A + 4),
               dict(w=_m(codes=A + 4)), dict(w=_m(scales=A + 2))):
        assert _call(L, _cfg(), **kw) == B.MOE_ERR_ALIGNMENT
    assert _call(L, _cfg(act=B.ACT["swiglu"]), w3=_m(scales=A + 8)) == B.MOE_ERR_ALIGNMENT


def test_pack_refusals(L):
    for fn in (lambda E, N, K, G, t, w, c, s: L.moe_q4_quantize(E, N, K, G, t, w, c, s, None),
               lambda E, N, K, G, t, w, c, s: L.moe_q4_dequantize(E, N, K, G, t, _m(c, s), w, None)):
        for args, want in [((0, 8, 32, 32, 0), 1), ((1, -8, 32, 32, 0), 1), ((1, 8, 0, 32, 0), 1),
                           ((1, 8, 32, 32, 2), 1), ((1, 8, 32, 32, -1), 1), ((1, 12, 32, 32, 0), 2),
                           ((1, 8, 40, 32, 0), 2), ((1, 8, 32, 40, 0), 2), ((1 << 20, 1 << 12, 32, 32, 0), 2),
                           ((1 << 10, 1 << 15, 1 << 16, 32, 0), 2), ((1, 8, (1 << 28) + 32, 32, 0), 2),
                           ((1, (1 << 28) + 8, 32, 32, 0), 2)]:
            assert fn(*args, A, A, A) == want, args
        ok = (1, 8, 32, 32, 1)
        for i in range(3):
            ptrs = [A, A, A]
            ptrs[i] = None
            assert fn(*ok, *ptrs) == B.MOE_ERR_INVALID_ARG
            ptrs[i] = A + 8
            assert fn(*ok, *ptrs) == B.MOE_ERR_ALIGNMENT
    assert L.moe_q4_dequantize(1, 8, 32, 32, 1, None, A, None) == B.MOE_ERR_INVALID_ARG


def _weights(**kw):
    w = B.moe_q4_weights()
    for n in ("w_gate", "b1", "b2", "logit_bias", "corr_bias"):
        setattr(w, n, A)
    for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        setattr(w, n, B.moe_q4_matrix(A, A))
    w.group = 32
    for n, v in kw.items():
        setattr(w, n, v)
    return w


def _layer_cfg(**kw):
    base = dict(T=4, D=64, F=32, E=8, k=2, act="swiglu", score="softmax", dtype="bf16", has_bias=False)
    base.update(kw)
    return B.make_config(**base)


def _decode(L, c, w, x=A, y=A, idx=A, gate=A, ws=A, nbytes=1 << 40):
    return L.moe_q4_decode(ctypes.byref(c), None if w is None else ctypes.byref(w), x, y, idx, gate, ws,
                           nbytes, None)


def _forward(L, c, w, x=A, y=A, ws=A, nbytes=1 << 40):
    return L.moe_q4_forward(ctypes.byref(c), None if w is None else ctypes.byref(w), x, y, ws, nbytes, None)


@pytest.mark.parametrize("call", [_decode, _forward])
def test_layer_refusals(L, call):
    bad, no = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
    c = _layer_cfg()
    for kw in (dict(dtype="f32"), dict(D=40), dict(F=40), dict(E=12), dict(k=9)):
        assert call(L, _layer_cfg(**kw), _weights()) == no, kw
    assert call(L, c, _weights(group=16)) == no
    assert call(L, _layer_cfg(T=-1), _weights()) == bad
    assert call(L, c, None) == bad
    assert call(L, c, _weights(w_gate=None)) == bad
    for n in ("w1", "w3", "w2"):
        assert call(L, c, _weights(**{n: B.moe_q4_matrix(None, A)})) == bad
        assert call(L, c, _weights(**{n: B.moe_q4_matrix(A, None)})) == bad
        assert call(L, c, _weights(**{n: B.moe_q4_matrix(A + 8, A)})) == B.MOE_ERR_ALIGNMENT
    for n in ("ws1", "ws3", "ws2"):
        assert call(L, _layer_cfg(n_shared=1), _weights(**{n: B.moe_q4_matrix(A, None)})) == bad
    biased = _layer_cfg(act="relu", has_bias=True)
    for n in ("b1", "b2"):
        assert call(L, biased, _weights(**{n: None})) == bad
        assert call(L, biased, _weights(**{n: A + 4})) == B.MOE_ERR_ALIGNMENT
    for kw in (dict(x=None), dict(y=None), dict(ws=None)):
        assert call(L, c, _weights(), **kw) == bad
    for kw in (dict(x=A + 8), dict(y=A + 8), dict(ws=A + 8)):
        assert call(L, c, _weights(), **kw) == B.MOE_ERR_ALIGNMENT
    assert call(L, c, _weights(), nbytes=64) == B.MOE_ERR_WORKSPACE_TOO_SMALL


def test_decode_keeps_the_few_token_limits(L):
    for kw in (dict(T=65), dict(D=16416), dict(F=8224), dict(F=4128, n_shared=2)):
        assert _decode(L, _layer_cfg(**kw), _weights()) == B.MOE_ERR_UNSUPPORTED


def test_workspace_grows_with_tokens():
    last = 0
    for T in list(range(0, 200, 7)) + [1000, 5000, 40000, 41000, 77824, 77825, 200000, 650000]:
        n = B.moe_q4_workspace_size(_layer_cfg(T=T))
        assert n >= last > -1
        last = n
    for kw in (dict(D=40), dict(F=40), dict(dtype="f32", E=8), dict(T=-1), dict(T=(1 << 30) + 8, k=1)):
        assert B.moe_q4_workspace_size(_layer_cfg(**kw)) == 0


def test_selftest_limits(L):
    cfg = _cfg()
    for limit in (0, -1, 2_000_000_001):
        assert L.moe_q4_selftest_wait_timeout(ctypes.byref(cfg), A, A, _m(), A, A, limit, None) == \
            B.MOE_ERR_INVALID_ARG


def test_calls_on_another_device(monkeypatch):
    """Tensors of a GPU that is not the current one never reach the library."""
    from types import SimpleNamespace
    calls = []

    class Fake:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or B.MOE_OK

    monkeypatch.setattr(B, "lib", lambda: Fake())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 77 + i)
    monkeypatch.setattr(B, "_ptr", lambda t: None)
    t = [SimpleNamespace(device=torch.device("cuda", i), numel=lambda: 0) for i in range(2)]
    m, c, w, cfg = B.moe_q4_matrix(), B.moe_q4_product_config(), B.moe_q4_weights(), _layer_cfg()
    for call in (lambda v: B.moe_q4_quantize(1, 8, 32, 32, "f32", v, v, v),
                 lambda v: B.moe_q4_dequantize(1, 8, 32, 32, "f32", m, v),
                 lambda v: B.moe_q4_product(c, v, v, m, None, None, v, v),
                 lambda v: B.moe_q4_selftest_wait_timeout(c, v, v, m, v, v, 5),
                 lambda v: B.moe_q4_decode(cfg, w, v, v, v), lambda v: B.moe_q4_forward(cfg, w, v, v, v),
                 lambda v: B.moe_q4_status(cfg, v)):
        n = len(calls)
        call(t[0])
        assert len(calls) == n + 1
        with pytest.raises(ValueError, match="cuda:1"):
            call(t[1])
        assert len(calls) == n + 1


def test_struct_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {n: getattr(B, n) for n in dir(B) if n.startswith("moe_q4_") and
               isinstance(getattr(B, n), type) and issubclass(getattr(B, n), ctypes.Structure)}
    assert structs
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_q4.h"', 'int main(void) {']
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += ['printf("%d\\n%d\\n", MOE_Q4_ACT_NONE, MOE_Q4_MAX_EXPERTS);', 'return 0; }']
    (tmp_path / "p.c").write_text("\n".join(lines))
    subprocess.run([cc, "-I", INCLUDE, str(tmp_path / "p.c"), "-o", str(tmp_path / "p")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for cls in structs.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want + [B.MOE_Q4_ACT_NONE, B.MOE_Q4_MAX_EXPERTS]


# ---- the Python classes

def _matrix(E=2, N=16, K=64, group=32):
    return Q4Matrix(torch.zeros(E, N, K // 2, dtype=torch.uint8),
                    torch.zeros(E, -(-K // group), N, dtype=torch.bfloat16), group)


def test_matrix_refusals():
    m = _matrix()
    assert m.shape == (2, 16, 64) and m.device.type == "cpu"
    codes, scales = m.codes, m.scales
    for c, s, g in [(codes, scales, 48), (codes[0], scales, 32), (codes.int(), scales, 32),
                    (codes, scales.float(), 32), (codes, scales, 64), (codes[:, :, :24], scales, 32),
                    (codes[:, :12].contiguous(), scales, 32), (codes.transpose(0, 1), scales, 32),
                    (codes, scales.transpose(1, 2).contiguous().transpose(1, 2), 32),
                    (codes[:0], scales[:0], 32), (codes.to("meta"), scales, 32)]:
        with pytest.raises(ValueError):
            Q4Matrix(c, s, g)
    with pytest.raises(AttributeError):
        m.codes = codes
    with pytest.raises(AttributeError):
        m.group = 64


def test_decoder_refusals():
    from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder
    from sparse_mixture_experts_softmax_gb300.q4_layer import Q4Layer
    g, up, down = torch.zeros(8, 64), _matrix(8, 32, 64), _matrix(8, 64, 32)
    for kw in (dict(w2=_matrix(8, 32, 64)), dict(w2=_matrix(8, 64, 32, 64)),
               dict(w2=torch.zeros(8, 64, 32, dtype=torch.bfloat16)), dict(w3=torch.zeros(8, 32, 64)),
               dict(w3=None), dict(w3=_matrix(8, 40, 64)), dict(n_shared=1),
               dict(n_shared=1, ws1=_matrix(1, 32, 64), ws3=_matrix(1, 32, 64), ws2=_matrix(1, 64, 64)),
               dict(w_gate=torch.zeros(8, 32)), dict(w1=torch.zeros(8, 32, 64).bfloat16())):
        args = dict(w_gate=g, w1=up, w2=down, w3=up, act="swiglu", k=2)
        args.update(kw)
        for cls in (MoEDecoder, Q4Layer):
            with pytest.raises(ValueError):
                cls(**args)
    with pytest.raises(ValueError, match="Q4Matrix"):        # plain weights make a decoder, not a Q4Layer
        Q4Layer(g, torch.zeros(8, 32, 64).bfloat16(), torch.zeros(8, 64, 32).bfloat16(), act="relu", k=2)
    layer = Q4Layer(g, up, down, w3=up, act="swiglu", k=2, max_tokens=3)
    for x in (torch.zeros(4, 64).bfloat16(), torch.zeros(3, 64), torch.zeros(3, 32).bfloat16()):
        with pytest.raises(ValueError):
            layer.forward(x)
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(3, 64).bfloat16(), torch.zeros(3, 64).bfloat16())
    with pytest.raises(ValueError, match="GPU"):
        layer.forward(torch.zeros(3, 64).bfloat16())
    with pytest.raises(AttributeError):
        layer.workspace = None
    with pytest.raises(ValueError):
        Q4Layer(g, up, down, w3=up, act="swiglu", k=2, max_tokens=0)


def test_quantize_refusals():
    for w, kw in [(torch.zeros(8, 32, dtype=torch.float16), {}), (torch.zeros(8, 40), {}),
                  (torch.zeros(12, 32), {}), (torch.zeros(32), {}), (torch.zeros(0, 8, 32), {}),
                  (torch.zeros(8, 32), dict(group=16)), (torch.zeros(32, 8).t(), {}),
                  (torch.zeros(8, 32), dict(out=_matrix())),
                  (torch.zeros(2, 16, 64), dict(group=64, out=_matrix()))]:
        with pytest.raises(ValueError):
            quantize(w, **kw)
    with pytest.raises(ValueError, match="GPU"):        # a CPU tensor never reaches the library
        quantize(torch.zeros(8, 32))
    with pytest.raises(ValueError, match="GPU"):
        _matrix().dequantize()
    with pytest.raises(ValueError):
        _matrix().dequantize(torch.float16)
    with pytest.raises(ValueError):
        _matrix().dequantize(out=torch.zeros(2, 16, 32))


def test_product_class_refusals():
    m = _matrix()
    for args, kw in [((m,), dict(act="silu")), ((m, m), dict(act="none")), ((m,), dict(act="swiglu")),
                     ((m, _matrix(N=24)), dict(act="swiglu")), ((m, _matrix(group=64)), dict(act="swiglu")),
                     ((_matrix(E=257),), {}), ((m, m), dict(act="swiglu", bias=torch.zeros(2, 16))),
                     ((m,), dict(bias=torch.zeros(2, 8))), ((m,), dict(bias=torch.zeros(2, 16).double()))]:
        with pytest.raises(ValueError):
            Q4Product(*args, **kw)
    p = Q4Product(m, bias=torch.zeros(2, 16), act="relu")
    x, off = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for xx, oo, out in [(x.float(), off, None), (x[:, :32], off, None), (x, off[:2], None),
                        (x, off.long(), None), (x[0], off, None), (x, off, torch.zeros(4, 16)),
                        (x, off, torch.zeros(5, 16, dtype=torch.bfloat16)),
                        (torch.zeros(4, 128, dtype=torch.bfloat16)[:, ::2], off, None)]:
        with pytest.raises(ValueError):
            p.forward(xx, oo, out)
    with pytest.raises(ValueError, match="GPU"):
        p.forward(x, off)
    with pytest.raises(AttributeError):
        p.shape = (1, 2, 3)


@pytest.mark.parametrize("D,F,n_shared", [(32, 8224, 0), (16416, 32, 0), (32, 4128, 2)])
def test_layer_past_the_few_token_limits(D, F, n_shared):
    """The layer for prompts takes what moe_q4_forward takes; its form for a few tokens is
    absent there, and says so."""
    from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder
    from sparse_mixture_experts_softmax_gb300.q4_layer import Q4Layer
    g, up, down = torch.zeros(8, D), _matrix(8, F, D), _matrix(8, D, F)
    args = dict(w3=up, act="swiglu", k=2, n_shared=n_shared)
    if n_shared:
        args.update(ws1=_matrix(1, n_shared * F, D), ws3=_matrix(1, n_shared * F, D),
                    ws2=_matrix(1, D, n_shared * F))
    with pytest.raises(B.MoEError):
        MoEDecoder(g, up, down, **args)
    layer = Q4Layer(g, up, down, max_tokens=3, **args)
    assert layer.decoder is None
    with pytest.raises(ValueError, match="use forward"):
        layer.decode(torch.zeros(3, D).bfloat16())
    with pytest.raises(ValueError, match="GPU"):
        layer.forward(torch.zeros(3, D).bfloat16())
    with pytest.raises(B.MoEError):                          # past moe_q4_forward's own
        Q4Layer(g, up, down, max_tokens=1 << 30, **args)

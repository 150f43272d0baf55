"""Refusals and sizes of the layer norm's entry points (host checks, no GPU)."""

import ctypes
import os

import pytest
import torch

from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.build import LIB, build_library
from sparse_mixture_experts_softmax_gb300.norm import LayerNorm, NormOut

A = 0x7f0000000000          # a fake aligned address: host checks never follow it
OK = dict(T=4, D=64, x_type="bf16", delta_type="f32", z_type="bf16", eps=1e-5)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB):
        build_library()
    return B.lib()


def _cfg(**kw):
    raw = {k: kw.pop(k) for k in ("raw_x", "raw_z", "raw_delta") if k in kw}
    c = B.make_norm_config(**dict(OK, **kw))
    c.x_type = raw.get("raw_x", c.x_type)
    c.z_type = raw.get("raw_z", c.z_type)
    c.delta_type = raw.get("raw_delta", c.delta_type)
    return c


def _fwd(L, c, x=A, delta=A, gamma=A, beta=A, h=A, z=A, mean=A, rstd=A):
    return L.moe_norm_forward(ctypes.byref(c) if c is not None else None, x, delta, gamma, beta, h,
                              z, mean, rstd, None)


def _bwd(L, c, h=A, dz=A, mean=A, rstd=A, gamma=A, dres=A, dx=A, dgamma=A, dbeta=A, ws=A,
         nbytes=1 << 40):
    return L.moe_norm_backward(ctypes.byref(c) if c is not None else None, h, dz, mean, rstd, gamma,
                               dres, dx, dgamma, dbeta, ws, nbytes, None)


def test_header_layout_matches(tmp_path):
    """The ctypes mirror against a C compiler's layout of the header."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_block.h"', 'int main(void){',
             'printf("%zu\\n", sizeof(moe_norm_config));']
    lines += [f'printf("%zu\\n", offsetof(moe_norm_config, {n}));'
              for n, _ in B.moe_norm_config._fields_]
    (tmp_path / "p.c").write_text("\n".join(lines + ["return 0;}"]))
    exe = str(tmp_path / "p")
    subprocess.run([cc, "-I", inc, str(tmp_path / "p.c"), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(B.moe_norm_config)] + \
        [getattr(B.moe_norm_config, n).offset for n, _ in B.moe_norm_config._fields_]


@pytest.mark.parametrize("kw", [dict(T=-1), dict(D=0), dict(D=-8), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(raw_x=2),
                                dict(raw_x=-1)])
def test_bad_configurations(L, kw):
    c = _cfg(**kw)
    assert _fwd(L, c) == B.MOE_ERR_INVALID_ARG
    assert _bwd(L, c) == B.MOE_ERR_INVALID_ARG
    assert B.moe_norm_workspace_size(c) == 0


@pytest.mark.parametrize("D", [16392, 8193, 9001, 1 << 20])
def test_unsupported_widths(L, D):
    c = _cfg(D=D)
    assert _fwd(L, c) == B.MOE_ERR_UNSUPPORTED
    assert _bwd(L, c) == B.MOE_ERR_UNSUPPORTED
    assert B.moe_norm_workspace_size(c) == 0


def test_forward_refusals(L):
    c = _cfg()
    assert _fwd(L, None) == B.MOE_ERR_INVALID_ARG
    assert _fwd(L, _cfg(raw_z=7)) == B.MOE_ERR_INVALID_ARG
    assert _fwd(L, _cfg(raw_delta=7)) == B.MOE_ERR_INVALID_ARG
    for name in ("x", "gamma", "z"):
        assert _fwd(L, c, **{name: None}) == B.MOE_ERR_INVALID_ARG
    assert _fwd(L, c, h=None) == B.MOE_ERR_INVALID_ARG           # a delta needs a place for h
    assert _fwd(L, c, delta=None) == B.MOE_ERR_INVALID_ARG       # h without a delta
    for name in ("x", "delta", "gamma", "beta", "h", "z", "mean", "rstd"):
        assert _fwd(L, c, **{name: A + 8}) == B.MOE_ERR_ALIGNMENT


def test_backward_refusals(L):
    c = _cfg()
    assert _bwd(L, None) == B.MOE_ERR_INVALID_ARG
    for name in ("h", "dz", "mean", "rstd", "gamma", "dx", "dgamma", "ws"):
        assert _bwd(L, c, **{name: None}) == B.MOE_ERR_INVALID_ARG
    for name in ("h", "dz", "mean", "rstd", "gamma", "dres", "dx", "dgamma", "dbeta", "ws"):
        assert _bwd(L, c, **{name: A + 4}) == B.MOE_ERR_ALIGNMENT
    need = B.moe_norm_workspace_size(c)
    assert need >= 2 * 64 * 4
    assert _bwd(L, c, nbytes=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL


def test_workspace_covers_one_row_and_none(L):
    assert B.moe_norm_workspace_size(_cfg(T=0)) > 0
    assert B.moe_norm_workspace_size(_cfg(T=1)) >= 2 * 64 * 4
    assert B.moe_norm_workspace_size(_cfg(T=1 << 30, D=16384)) < 1 << 30


def test_python_refusals(L):
    gamma = torch.ones(16)
    with pytest.raises(ValueError):
        LayerNorm(gamma.double())
    with pytest.raises(ValueError):
        LayerNorm(gamma, torch.zeros(15))
    n = LayerNorm(gamma, x_dtype="f32")
    x = torch.zeros(3, 16)
    for bad in (torch.zeros(16), torch.zeros(3, 17), x.bfloat16(), torch.zeros(16, 3).t()):
        with pytest.raises(ValueError):
            n.forward(bad)
    with pytest.raises(ValueError):
        n.forward(x, torch.zeros(2, 16))
    with pytest.raises(ValueError):
        n.forward(x, torch.zeros(3, 16, dtype=torch.float16))
    with pytest.raises(ValueError):
        n.forward(x, out=NormOut(x, x, None, None))          # h without a delta
    with pytest.raises(ValueError):
        n.backward(x, x, torch.zeros(2), torch.zeros(3))
    with pytest.raises(ValueError):
        n.backward(x.bfloat16(), x, torch.zeros(3), torch.zeros(3))
    with pytest.raises(ValueError):
        n.backward(x, x, torch.zeros(3), torch.zeros(3), dres=torch.zeros(3, 15))


def test_workspace_of_any_rows(L):
    """The workspace for the most rows holds every smaller call's."""
    for D in (1, 7, 64, 4096, 8191, 16384):
        most = B.moe_norm_workspace_size(_cfg(T=2**31 - 1, D=D))
        sizes = [B.moe_norm_workspace_size(_cfg(T=T, D=D)) for T in (0, 1, 17, 303, 4096, 1 << 20)]
        assert 0 < max(sizes) <= most and sizes == sorted(sizes)


def test_python_refuses_host_tensors(L):
    n, x = LayerNorm(torch.ones(16)), torch.zeros(3, 16)
    with pytest.raises(ValueError, match="GPU"):
        n.forward(x)
    with pytest.raises(ValueError, match="GPU"):
        n.backward(x, x, torch.zeros(3), torch.zeros(3))


def test_what_a_norm_is_made_of_stays(L):
    """Calls pass addresses and configurations taken once: replacing what they were
    taken from would leave them at freed memory or with the old values."""
    n = LayerNorm(torch.ones(16), torch.zeros(16))
    n.beta = n.beta             # (as ``n.beta += t`` ends)
    for name, value in (("gamma", torch.ones(16)), ("beta", None), ("D", 8), ("eps", 1e-6),
                        ("x_type", torch.bfloat16), ("z_type", torch.bfloat16),
                        ("device", torch.device("meta"))):
        with pytest.raises(AttributeError, match=name):
            setattr(n, name, value)
    n.gamma *= 2                # in place is how they are trained
    assert float(n.gamma[0]) == 2.0

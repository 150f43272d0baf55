"""The layer norm of the residual block (moe_norm_forward, moe_norm_backward)
against its formulas in 64 bits: widths that end inside a vector, a warp and a
block, every type, in-place outputs, rows of equal values, and the gradients
against differences.

Tolerances.  z is computed in fp32 from the exact row and rounded once: for an
output type of step eps the error is at most eps/2 |z| plus the fp32 part.  The
fp32 part of a row of D values: mean and rstd come from sums of D terms in a
tree of depth at most log2(1024) + 16 adds, each 2^-24; with the handful of
products behind them the relative error of xh stays under 40 * 2^-24 = 2.4e-6 of
the largest |h - mean| rstd and |mean| rstd of the row.
"""

import numpy as np
import pytest
import torch

from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.norm import LayerNorm, NormGrads, NormOut

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
F32 = 40 * 2.0 ** -24
EPS = 1e-5


def _stream(T, D, x, seed=0, offset=0.25, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, D, generator=g) * spread + offset).to(DT[x]).cuda()


def _params(D, seed=1, beta=True):
    g = torch.Generator().manual_seed(seed)
    gamma = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    return gamma, (0.3 * torch.randn(D, generator=g)).cuda() if beta else None


def _reference(h, gamma, beta, eps=EPS):
    v = h.double()
    mean = v.mean(1)
    rstd = 1 / ((v - mean[:, None]).square().mean(1) + eps).sqrt()
    xh = (v - mean[:, None]) * rstd[:, None]
    z = xh * gamma.double() + (beta.double() if beta is not None else 0)
    return mean, rstd, xh, z


def _check_forward(n, h, r, z_type, gamma, beta):
    mean, rstd, xh, z = _reference(h, gamma, beta, n.eps)
    amp = torch.maximum(xh.abs().amax(1), mean.abs() * rstd)[:, None]
    slack = F32 * amp * gamma.double().abs() + F32 * z.abs() + HALF[z_type] * z.abs()
    bad = (r.z.double() - z).abs() > slack
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"
    if r.mean is not None:
        scale = h.double().abs().amax(1)
        assert ((r.mean.double() - mean).abs() <= F32 * scale).all()
        # the variance's error is relative to itself and the mean's error squared
        assert ((r.rstd.double() - rstd).abs() <= F32 * (1 + amp[:, 0]) * rstd).all()


@pytest.mark.parametrize("x,z,delta", [("f32", "f32", None), ("f32", "bf16", "f32"),
                                       ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                       ("bf16", "bf16", None), ("f32", "f32", "bf16")])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 8), (3, 7), (1, 4096), (5, 255), (9, 256), (17, 264),
                                 (2, 1023), (700, 520), (33, 2056), (4, 8192), (3, 8191),
                                 (2, 8200), (2, 16384)])
def test_forward(T, D, x, z, delta):
    gamma, beta = _params(D)
    h0 = _stream(T, D, x)
    d = _stream(T, D, delta, seed=5, offset=0.0, spread=0.5) if delta else None
    n = LayerNorm(gamma, beta, x_dtype=x, z_dtype=z, eps=EPS)
    keep = h0.clone()
    r = n.forward(h0, d)
    torch.cuda.synchronize()
    assert torch.equal(h0, keep)
    if delta:
        want = (h0.float() + d.float()).to(DT[x])     # one fp32 sum, rounded: bit for bit
        assert torch.equal(r.h, want)
    else:
        assert r.h is None
    _check_forward(n, r.h if delta else h0, r, z, gamma, beta)


def test_forward_without_stats_and_shift():
    gamma, _ = _params(72)
    h = _stream(6, 72, "bf16")
    n = LayerNorm(gamma, None, x_dtype="bf16", z_dtype="f32")
    r = n.forward(h, stats=False)
    assert r.mean is None and r.rstd is None
    full = n.forward(h)
    assert torch.equal(full.z, r.z)
    _check_forward(n, h, full, "f32", gamma, None)


def test_forward_serving_buffers():
    """Without statistics and ``out`` the outputs are the norm's own buffers; a
    stream that is one of them is updated in place; sizes may alternate."""
    gamma, beta = _params(96)
    n = LayerNorm(gamma, beta, "bf16", "bf16")
    for T in (3, 1, 3):
        x, d = _stream(T, 96, "bf16", seed=T), _stream(T, 96, "bf16", seed=T + 7)
        want = n.forward(x, d)
        r = n.forward(x, d, stats=False)
        assert torch.equal(r.h, want.h) and torch.equal(r.z, want.z)
        nxt = n.forward(want.h, d)
        again = n.forward(r.h, d, stats=False)
        assert again.h is r.h and torch.equal(again.h, nxt.h) and torch.equal(again.z, nxt.z)
        alone = n.forward(x, stats=False)
        assert alone.h is None and torch.equal(alone.z, n.forward(x).z)


def test_forward_in_place_stream():
    gamma, beta = _params(136)
    x, d = _stream(11, 136, "f32"), _stream(11, 136, "f32", seed=9)
    n = LayerNorm(gamma, beta)
    fresh = n.forward(x, d)
    own = x.clone()
    out = NormOut(own, torch.empty_like(fresh.z), torch.empty_like(fresh.mean),
                  torch.empty_like(fresh.rstd))
    r = n.forward(own, d, out=out)
    assert r.h is own and torch.equal(own, fresh.h) and torch.equal(r.z, fresh.z)


def test_large_offset_and_equal_rows():
    """A row far from zero keeps its spread (the variance is no difference of
    large squares), and a row of equal values gives z = beta exactly."""
    gamma, beta = _params(512)
    h = _stream(4, 512, "f32", offset=3000.0)
    h[2] = 7.0
    n = LayerNorm(gamma, beta, eps=EPS)
    r = n.forward(h)
    assert torch.equal(r.z[2], beta)
    _check_forward(n, h[:2].contiguous(), NormOut(None, r.z[:2], r.mean[:2], r.rstd[:2]), "f32",
                   gamma, beta)


def test_non_finite_rows_stay_in_their_row():
    gamma, beta = _params(264)
    h = _stream(5, 264, "bf16")
    clean = LayerNorm(gamma, beta, "bf16", "bf16").forward(h)
    h2 = h.clone()
    h2[1, 3] = float("inf")
    h2[3, 200] = float("nan")
    r = LayerNorm(gamma, beta, "bf16", "bf16").forward(h2)
    assert torch.isnan(r.z[1]).all() and torch.isnan(r.z[3]).all()
    for t in (0, 2, 4):
        assert torch.equal(r.z[t], clean.z[t])


def _backward_case(T, D, x, res=True, beta=True, seed=3):
    gamma, b = _params(D, beta=beta)
    h = _stream(T, D, x, seed=seed)
    n = LayerNorm(gamma, b, x_dtype=x, z_dtype="f32", eps=EPS)
    f = n.forward(h)
    g = torch.Generator().manual_seed(seed + 1)
    dz = torch.randn(T, D, generator=g).cuda()
    dres = torch.randn(T, D, generator=g).cuda() if res else None
    return n, h, f, dz, dres


def _check_backward(n, h, f, dz, dres, out):
    T, D = h.shape
    m, r = f.mean.double()[:, None], f.rstd.double()[:, None]
    xh = (h.double() - m) * r
    g = dz.double() * n.gamma.double()
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2) + (dres.double() if dres is not None else 0)
    amp = torch.maximum(xh.abs(), m.abs() * r)
    # fp32 error of each term of dx, as in the module docstring; c1 and c2 are
    # bounded by the row's largest products
    gm = g.abs().amax(1, keepdim=True)
    slack = F32 * (r * gm * (1 + amp + amp.amax(1, keepdim=True) ** 2) + dx.abs())
    assert ((out.dx.double() - dx).abs() <= slack).all()
    # dgamma, dbeta: at most ceil(T/blocks) sequential adds, then a tree of the
    # partial sums; each add is off by 2^-24 of a sum of at most sum |terms|
    steps = 8 + T / max(1, min(T, 152)) + 40
    tol = steps * 2.0 ** -24
    terms = (dz.double() * xh).abs().sum(0) + F32 * (dz.double().abs() * amp).sum(0) / tol
    assert ((out.dgamma.double() - (dz.double() * xh).sum(0)).abs() <= tol * terms).all()
    if out.dbeta is not None:
        assert ((out.dbeta.double() - dz.double().sum(0)).abs()
                <= tol * dz.double().abs().sum(0)).all()


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 8), (3, 7), (1, 4096), (5, 255), (9, 256), (5000, 64),
                                 (17, 264), (400, 1023), (700, 520), (1300, 2056), (4, 8192),
                                 (3, 8191), (200, 8200), (2, 16384)])
def test_backward(T, D, x):
    n, h, f, dz, dres = _backward_case(T, D, x)
    out = NormGrads(*[t.clone() for t in n.backward(dz, h, f.mean, f.rstd, dres=dres)])
    _check_backward(n, h, f, dz, dres, out)
    again = n.backward(dz, h, f.mean, f.rstd, dres=dres)
    assert again.dgamma is n.dgamma and again.dbeta is n.dbeta
    for a, b in zip(out, again):
        assert torch.equal(a, b)        # fixed-order sums: the same bits


@pytest.mark.parametrize("res,beta", [(False, True), (True, False), (False, False)])
def test_backward_optional_parts(res, beta):
    n, h, f, dz, dres = _backward_case(50, 328, "bf16", res, beta)
    out = n.backward(dz, h, f.mean, f.rstd, dres=dres)
    assert (out.dbeta is None) == (not beta)
    _check_backward(n, h, f, dz, dres, out)


@pytest.mark.parametrize("onto", ["dz", "dres"])
def test_backward_in_place(onto):
    n, h, f, dz, dres = _backward_case(37, 2048, "f32")
    want = n.backward(dz, h, f.mean, f.rstd, dres=dres)
    buf = dz if onto == "dz" else dres
    out = NormGrads(buf, torch.empty_like(want.dgamma), torch.empty_like(want.dbeta))
    n.backward(dz, h, f.mean, f.rstd, dres=dres, out=out)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_backward_against_differences():
    """Central differences of L = sum(w z) + sum(dres h) in 64 bits: the second
    difference's error is h^2 times the third derivative, about 1e-8 at
    h = 1e-4, so 1e-5 of the gradient's size separates a right gradient from a
    wrong term."""
    T, D = 3, 24
    n, h, f, dz, dres = _backward_case(T, D, "f32")
    out = n.backward(dz, h, f.mean, f.rstd, dres=dres)

    def loss(hv, gamma, beta):
        z = _reference(hv, gamma, beta)[3]
        return float((dz.double() * z).sum() + (dres.double() * hv).sum())

    base = [h.double(), n.gamma.double(), n.beta.double()]
    for k, grad in enumerate((out.dx, out.dgamma, out.dbeta)):
        flat = grad.double().reshape(-1).cpu()
        for i in range(0, flat.numel(), 5):
            hi, lo = [b.clone() for b in base], [b.clone() for b in base]
            hi[k].view(-1)[i] += 1e-4
            lo[k].view(-1)[i] -= 1e-4
            num = (loss(*hi) - loss(*lo)) / 2e-4
            assert abs(num - float(flat[i])) <= 1e-5 * (1 + abs(num)), (k, i)


def test_zero_rows():
    n, h, f, dz, dres = _backward_case(4, 40, "f32")
    e = torch.empty(0, 40, device="cuda")
    r = n.forward(e, e)
    assert r.z.shape == (0, 40)
    out = NormGrads(e, torch.full_like(n.gamma, 3), torch.full_like(n.gamma, 3))
    n.backward(e, e, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), out=out)
    assert not out.dgamma.any() and not out.dbeta.any()


def test_on_a_side_stream_and_in_a_graph():
    n, h, f, dz, dres = _backward_case(300, 1024, "bf16")
    want, wantf = n.backward(dz, h, f.mean, f.rstd, dres=dres), n.forward(h)
    s = torch.cuda.Stream()
    out = NormGrads(torch.empty_like(dz), torch.empty_like(n.gamma), torch.empty_like(n.gamma))
    outf = NormOut(None, torch.empty_like(wantf.z), None, None)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        n.forward(h, out=outf)
        n.backward(dz, h, f.mean, f.rstd, dres=dres, out=out)
    out.dx.zero_()
    outf.z.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outf.z, wantf.z)
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    with torch.cuda.stream(s):
        r = n.forward(h)
    s.synchronize()
    assert torch.equal(r.z, wantf.z)


def test_more_than_2_31_elements():
    """Row offsets pass 32 bits: the last rows are checked."""
    D = 16384
    T = (1 << 31) // D + 3
    gamma, beta = _params(D)
    h = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    h.normal_(generator=torch.Generator("cuda").manual_seed(1))
    n = LayerNorm(gamma, beta, "bf16", "bf16")
    r = n.forward(h)
    tail = slice(T - 4, T)
    _check_forward(n, h[tail].contiguous(), NormOut(None, r.z[tail], r.mean[tail], r.rstd[tail]),
                   "bf16", gamma, beta)


def test_graphs_keep_their_buffers():
    """A graph of a few rows, or of a small backward pass, still writes to memory
    of the norm's own after calls of other sizes."""
    gamma, beta = _params(96)
    n = LayerNorm(gamma, beta)
    x, dz = _stream(1, 96, "f32"), _stream(1, 96, "f32", seed=3)
    want = n.forward(x)
    n.forward(x, stats=False)
    grads = n.backward(dz, x, want.mean, want.rstd)
    dx, dgamma = grads.dx.clone(), grads.dgamma.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = n.forward(x, stats=False)
        b = n.backward(dz, x, want.mean, want.rstd, out=grads)
    held = n.workspace.data_ptr(), r.z.data_ptr()
    for T in (2, 65, 5000):
        big = _stream(T, 96, "f32", seed=T)
        s = n.forward(big)
        assert torch.equal(n.forward(big, stats=False).z, s.z)
        n.backward(big, big, s.mean, s.rstd)
    assert held == (n.workspace.data_ptr(), n.forward(x, stats=False).z.data_ptr())
    others = [torch.full((1, 96), 7.0, device="cuda") for _ in range(64)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.z, want.z) and torch.equal(b.dx, dx) and torch.equal(b.dgamma, dgamma)
    assert all(bool((o == 7.0).all()) for o in others)


def test_parameter_storage_is_kept():
    """Replacing a parameter's storage neither frees nor changes what the norm reads."""
    gamma, beta = _params(64)
    p = torch.nn.Parameter(gamma.clone())
    n, x = LayerNorm(p, beta), _stream(5, 64, "f32")
    want = LayerNorm(gamma, beta).forward(x).z
    p.data = torch.zeros_like(gamma)
    assert torch.equal(n.forward(x).z, want)


def test_the_norms_own_parameters_keep_their_storage():
    """So does replacing the storage of the norm's own attribute."""
    gamma, beta = _params(64)
    n, x = LayerNorm(gamma.clone(), beta), _stream(5, 64, "f32")
    want = n.forward(x).z
    n.gamma.data = torch.zeros_like(gamma)
    others = [torch.zeros(64, device="cuda") for _ in range(16)]     # where a freed one would be
    assert torch.equal(n.forward(x).z, want) and len(others) == 16


def test_direct_bindings():
    """The binding's functions, as a program without the class calls them."""
    T, D = 21, 264
    gamma, beta = _params(D)
    h, d = _stream(T, D, "bf16"), _stream(T, D, "f32", seed=2, offset=0.0)
    n = LayerNorm(gamma, beta, "bf16", "bf16")
    want = n.forward(h, d)
    cfg = B.make_norm_config(T, D, x_type="bf16", delta_type="f32", z_type="bf16")
    got = NormOut(*[torch.empty_like(t) for t in want])
    B.moe_norm_forward(cfg, h, d, gamma, beta, got.h, got.z, got.mean, got.rstd)
    assert B.moe_last_launch_count() == 1
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    dz, dres = _stream(T, D, "f32", seed=4), _stream(T, D, "f32", seed=5)
    want = n.backward(dz, got.h, got.mean, got.rstd, dres=dres)
    out = NormGrads(*[torch.empty_like(t) for t in want])
    ws = torch.empty(B.moe_norm_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.moe_norm_backward(cfg, got.h, dz, got.mean, got.rstd, gamma, dres, out.dx, out.dgamma,
                        out.dbeta, ws, stream=s)
    assert B.moe_last_launch_count() == 2
    s.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)

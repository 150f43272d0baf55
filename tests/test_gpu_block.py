"""The pre-norm residual block: norm, layer and both backward passes against
their formulas in 64 bits, and serving against training.

Tolerances.  fp32 blocks: the layer's own parity tolerance (1e-4 of a tensor's
largest value) on every output; the norm in front adds a few 2^-24.  bf16 blocks
hold the layer's 2e-2.  A served token against the trained layer's: the training
forward rounds hidden rows, Y_e and (here) nothing else to bf16, the served one
its y: three half steps of 2^-8.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

import workloads as W
from oracle import moe_oracle as O
from sparse_mixture_experts_softmax_gb300.block import MoEBlock
from sparse_mixture_experts_softmax_gb300.norm import LayerNorm
from tests.moe_cases import TOL, assert_close, make_layer, np64, oracle_config, oracle_inputs

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _block(name, T, seed, x_dtype):
    wl = W.WORKLOADS[name].with_tokens(T)
    inp = W.make_inputs(wl, seed=seed, with_target=False)
    inp["target"] = None
    g = torch.Generator().manual_seed(seed + 5)
    gamma = (1 + 0.2 * torch.randn(wl.D, generator=g)).cuda()
    beta = (0.1 * torch.randn(wl.D, generator=g)).cuda()
    norm = LayerNorm(gamma, beta, x_dtype=x_dtype, z_dtype=wl.dtype, eps=EPS)
    return wl, inp, MoEBlock(norm, make_layer(wl, inp))


def _norm64(h, gamma, beta):
    m = h.mean(1, keepdims=True)
    r = 1 / np.sqrt(((h - m) ** 2).mean(1, keepdims=True) + EPS)
    xh = (h - m) * r
    return xh, r, xh * gamma + beta


@pytest.mark.parametrize("name,T,x_dtype", [("dense_f32", 96, "f32"), ("grouped", 130, "bf16"),
                                            ("grouped_shared", 64, "f32"), ("tiny", 64, "f32")])
def test_block_forward_and_gradients(name, T, x_dtype):
    wl, inp, block = _block(name, T, 3, x_dtype)
    g = torch.Generator().manual_seed(11)
    dt = torch.bfloat16 if x_dtype == "bf16" else torch.float32
    h0 = torch.randn(T, wl.D, generator=g).to(dt).cuda()
    delta = (0.3 * torch.randn(T, wl.D, generator=g)).cuda()
    dout = torch.randn(T, wl.D, generator=g).cuda() / T
    state, y = block.forward(h0, delta)
    dx = block.backward(state, dout)
    torch.cuda.synchronize()

    assert torch.equal(state.h, (h0.float() + delta).to(dt))
    cfg = oracle_config(wl)
    w, _, _, _ = oracle_inputs(wl, inp)
    gamma, beta = np64(block.norm.gamma), np64(block.norm.beta)
    xh, r, z = _norm64(np64(state.h), gamma, beta)
    assert_close("z", np64(state.z), z, 2.0 ** -8 if wl.dtype == "bf16" else 1e-6)
    # the layer's part from the z that it read (a bf16 z is a rounding of the formula's)
    zin = np64(state.z)
    st = O.forward(cfg, w, zin, block.layer.routing()["idx"].cpu().numpy())
    tol = TOL[wl.dtype]
    assert_close("y", np64(y), st["y"], tol)
    gr = O.backward(cfg, w, zin, st, np64(dout))
    dz, do = gr["dx"], np64(dout)
    gg = dz * gamma
    want_dx = do + r * (gg - gg.mean(1, keepdims=True) - xh * (gg * xh).mean(1, keepdims=True))
    assert_close("dx", np64(dx), want_dx, tol)
    assert_close("dgamma", np64(block.norm.dgamma), (dz * xh).sum(0), tol)
    assert_close("dbeta", np64(block.norm.dbeta), dz.sum(0), tol)
    for key in ("dw_gate", "dw1", "dw2"):
        assert_close(key, np64(getattr(block.layer, key)), gr[key], tol)


@pytest.mark.parametrize("name", ["grouped", "grouped_cb", "grouped_shared", "dense_bf16"])
def test_block_serves_what_it_trains(name):
    wl, inp, block = _block(name, 40, 4, "bf16")
    g = torch.Generator().manual_seed(2)
    h0 = torch.randn(40, wl.D, generator=g).bfloat16().cuda()
    delta = (0.3 * torch.randn(40, wl.D, generator=g)).cuda()
    state, y = block.forward(h0, delta)
    h, ys = block.decode(h0, delta)
    assert torch.equal(h, state.h)
    same = (block.decoder.idx == block.layer.routing()["idx"]).all(1)
    assert int(same.sum()) >= 38
    err = (ys.float() - y)[same].abs().max() / y.abs().max()
    assert err <= 3 * 2.0 ** -8
    assert block.decoder.status() == 0


def test_block_refusals():
    wl, inp, block = _block("tiny", 64, 1, "f32")
    with pytest.raises(ValueError):
        MoEBlock(LayerNorm(torch.ones(16, device="cuda")), block.layer)
    with pytest.raises(ValueError):
        MoEBlock(LayerNorm(torch.ones(wl.D, device="cuda"), z_dtype="bf16"), block.layer)


def test_example_runs():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "prenorm_blocks.py")
    spec = importlib.util.spec_from_file_location("prenorm_blocks", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, err = mod.main(6)
    assert losses[-1] < losses[0]
    assert err <= 2 * 3 * 2.0 ** -8        # two blocks


@pytest.mark.parametrize("how", ["attribute", "data"])
def test_block_does_not_serve_replaced_weights(how):
    """The decoder reads the storage that the layer's tensors had when it was made:
    weights trained in place are served, others are refused, not ignored."""
    wl, inp, block = _block("grouped_cb", 16, 6, "bf16")
    h0 = torch.randn(4, wl.D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    y = block.decode(h0)[1].clone()
    block.layer.w2_lp.mul_(2)
    assert torch.equal(block.decode(h0)[1], 2 * y)
    for name in ("w2_lp", "corr_bias"):
        old = getattr(block.layer, name)
        if how == "attribute":
            setattr(block.layer, name, old.clone())
        else:
            keep, old.data = old.data, old.clone()
        with pytest.raises(ValueError, match=name):
            block.decode(h0)
        if how == "attribute":
            setattr(block.layer, name, old)
        else:
            old.data = keep
    assert torch.equal(block.decode(h0)[1], 2 * y)
    again = MoEBlock(block.norm, block.layer)
    assert torch.equal(again.decode(h0)[1], 2 * y)

"""The MoE layer on 4-bit expert weights (moe_q4_decode, moe_q4_forward, Q4Layer, Q4Block)
against the float64 oracle on the weights that the codes stand for.

Tolerances.  The few-token layer: those of the layer on bf16 weights (tests/test_gpu_decode.py;
the weights are exact bf16 values, the sums no longer).  The prompts' layer: the training
forward's 2e-2 of a tensor's largest value (hidden activations, the experts' outputs and
the shared branch's are rounded to bf16 there as well)."""

import dataclasses

import numpy as np
import pytest
import torch

import workloads as W
from oracle import moe_oracle as O
from sparse_mixture_experts_softmax_gb300.block import Q4Block
from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder
from sparse_mixture_experts_softmax_gb300.norm import LayerNorm
from sparse_mixture_experts_softmax_gb300.q4 import Q4Matrix, quantize
from sparse_mixture_experts_softmax_gb300.q4_layer import Q4Layer
from tests.moe_cases import (TOL, assert_close, device_x, make_layer, np64, oracle_config,
                             oracle_inputs, validated_routing)
from tests.test_gpu_decode import _check, _inputs, _wl

pytestmark = pytest.mark.gpu

NAMES = ("w1", "w3", "w2", "ws1", "ws3", "ws2")


def _quantized(wl, seed, group):
    """Inputs whose expert weights are the values of 4-bit matrices, and the matrices."""
    inp = _inputs(wl, seed)
    ms = {}
    for n in NAMES:
        if inp.get(n) is None:
            continue
        ms[n] = quantize(inp[n].cuda(), group)
        v = ms[n].dequantize(torch.float32).cpu().reshape(inp[n].shape)
        inp[n], inp[n + "_bf16"] = v, v.bfloat16()
    return inp, ms


def _args(wl, inp, ms):
    c = lambda t: None if t is None else t.cuda().contiguous()  # noqa: E731
    return dict(w_gate=c(inp["w_gate"]), b1=c(inp["b1"]), b2=c(inp["b2"]), k=wl.k, act=wl.act,
                score=wl.score, n_groups=wl.n_groups, topk_groups=wl.topk_groups,
                logit_bias=c(inp["logit_bias"]), corr_bias=c(inp["corr_bias"]), n_shared=wl.n_shared,
                capacity_factor=wl.capacity_factor, **ms)


CASES = {
    "gelu_nobias": (32, dict(act="gelu_tanh", D=512, F=288, E=16, k=3)),
    "relu_bias": (64, dict(act="relu", has_bias=True, D=288, F=544, k=4)),
    "gelu_bias": (128, dict(act="gelu_tanh", has_bias=True, D=160, F=96, k=2)),
    "swiglu": (64, dict(D=1024, F=704, E=16, k=4)),
    "swiglu_short_group": (128, dict(D=1056, F=736, E=8, k=2)),
    "grouped_sigmoid": (32, dict(score="sigmoid", n_groups=8, topk_groups=4, E=64, k=6, D=256, F=96)),
    "corrected": (32, dict(score="sigmoid", n_groups=4, topk_groups=2, E=32, k=4, corr_bias_scale=0.1)),
    "shared": (64, dict(n_shared=2, E=16, k=2, D=352, F=224)),
    "skewed_empty": (32, dict(E=16, k=4, zipf_skew=1.2, zipf_empty=4, D=128, F=160)),
    "smallest": (32, dict(D=32, F=32, E=8, k=1)),
    "every_expert": (128, dict(E=8, k=8, D=96, F=64)),
    "capacity": (64, dict(E=8, k=2, D=128, F=64, capacity_factor=0.5)),
}


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("name", sorted(CASES))
def test_decode(name, T):
    group, kw = CASES[name]
    wl = _wl(T=T, **kw)
    inp, ms = _quantized(wl, T, group)
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=T)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("group,kw", [
    (64, dict(T=33, D=4096, F=64, E=8)), (32, dict(T=48, D=512, F=704, E=8, k=8)),
    (128, dict(T=40, D=4096, F=1024, E=8, k=4, n_shared=1)), (32, dict(T=64, D=32, F=32, E=256, k=32)),
    (32, dict(T=1, D=32, F=8192, E=8)), (128, dict(T=1, D=16384, F=32, E=8)),
    (64, dict(T=20, D=64, F=8192, E=8, act="relu")), (128, dict(T=3, D=4096, F=2048, E=16, k=8)),
])
def test_decode_sizes(group, kw):
    wl = _wl(**kw)
    inp, ms = _quantized(wl, 3, group)
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=wl.T)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


def test_decode_every_code_and_eight_bit_scales():
    """Codes of 0 to 15 and scales of eight bits: weights are the rounded products."""
    from tests import q4_cases as C
    wl = _wl(T=12, D=320, F=160, E=8, k=2)
    inp = _inputs(wl, 1)
    rng, ms = np.random.default_rng(2), {}
    for n in ("w1", "w3", "w2"):
        E, N, K = inp[n].shape
        codes, scales = C.random_matrix(rng, E, N, K, 64, five_bits=False)
        ms[n] = C.device_matrix(codes, scales, 64)
        v = torch.from_numpy(C.weights(codes, scales, 64)).float()
        inp[n], inp[n + "_bf16"] = v, v.bfloat16()
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=wl.T)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("T", [3, 4])
@pytest.mark.parametrize("name", sorted(CASES))
def test_decode_up_to_four_tokens(name, T):
    test_decode(name, T)


@pytest.mark.parametrize("T,kw", [(4, dict(D=32, F=8192, E=8, k=8)), (4, dict(D=16384, F=32, E=8, k=8)),
                                  (4, dict(D=4096, F=1024, E=8, k=4, n_shared=2)),
                                  (2, dict(D=32, F=32, E=256, k=32)), (4, dict(D=4096, F=4096, E=8, k=2))])
def test_decode_up_to_four_tokens_sizes(T, kw):
    wl = _wl(T=T, **kw)
    inp, ms = _quantized(wl, 5, 32)
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=T)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("T", [1, 4, 7, 12])
@pytest.mark.parametrize("up,down", [(2.0 ** 20, 2.0 ** -24), (2.0 ** -40, 2.0 ** 44), (2.0 ** -100, 2.0 ** 100)])
def test_decode_scales_of_any_size(T, up, down):
    """Scales of both projections on either side of what the kernel widens the short way;
    ReLU keeps the layer's scale."""
    from tests import q4_cases as C
    wl = _wl(T=T, D=320, F=160, E=8, k=2, act="relu")
    inp = _inputs(wl, 1)
    rng, ms = np.random.default_rng(2), {}
    for n, times in (("w1", up), ("w2", down)):
        E, N, K = inp[n].shape
        codes, scales = C.random_matrix(rng, E, N, K, 64, five_bits=False)
        scales = C.bf16(scales * times)
        ms[n] = C.device_matrix(codes, scales, 64)
        v = torch.from_numpy(C.weights(codes, scales, 64)).float()
        inp[n], inp[n + "_bf16"] = v, v.bfloat16()
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=wl.T)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("T", [1, 4, 6, 20])
def test_decode_infinite_scale(T):
    """An infinite and a NaN scale of the down projection stay in their outputs."""
    wl = _wl(T=T, D=96, F=160, E=8, k=8)
    inp, ms = _quantized(wl, 3, 32)
    m = ms["w2"]
    m.codes[m.codes == 0x88] = 0x99              # no weight of zero in either place of a byte
    codes = m.codes.cpu().numpy()
    codes[(codes & 15) == 8] += 1
    codes[(codes >> 4) == 8] += 16
    m.codes.copy_(torch.from_numpy(codes))
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=T)
    x = device_x(wl, inp)
    want = d.decode(x).clone()
    m.scales[:, 2, 5] = float("inf")
    m.scales[:, 4, 70] = float("nan")
    got = d.decode(x)
    rest = [i for i in range(96) if i not in (5, 70)]
    assert torch.equal(got[:, rest], want[:, rest]) and bool(want.isfinite().all())
    assert not bool(got[:, 5].isfinite().any()) and bool(got[:, 70].isnan().all())


def _forward_want(wl, inp, layer, x, idx_from):
    """The oracle's y with the kernel's choice between nearly equal experts."""
    cfg = oracle_config(wl)
    w, _, x64, _ = oracle_inputs(wl, inp)
    scores = O.router_scores(cfg, O.router_logits(x64, w["w_gate"], w["logit_bias"]))
    idx = validated_routing(cfg, scores, idx_from, corr_bias=w["corr_bias"])
    return O.forward(cfg, w, x64, idx)["y"]


def _routing_of(layer, T, k, E):
    """idx [T, k] of the last forward, from its workspace (after status and scores)."""
    at = 256 + -(-T * E * 4 // 256) * 256
    return layer.workspace[at:at + T * k * 4].view(torch.int32).view(T, k).cpu().numpy()


@pytest.mark.parametrize("T", [1, 7, 64, 130, 777])
@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name, T):
    group, kw = CASES[name]
    wl = _wl(T=T, **kw)
    inp, ms = _quantized(wl, T, group)
    layer = Q4Layer(**_args(wl, inp, ms), max_tokens=T + 5)
    x = device_x(wl, inp)
    y = layer.forward(x)
    assert layer.status() == 0
    want = _forward_want(wl, inp, layer, x, _routing_of(layer, T, wl.k, wl.E))
    assert_close("y", np64(y), want, TOL["bf16"])


def test_from_layer_prompt_then_tokens():
    """A trained layer's 4-bit form: prompts, then tokens, agree with each other, and
    follow the layer's further training."""
    wl = dataclasses.replace(W.WORKLOADS["grouped_shared"].with_tokens(96), D=512, F=256)
    inp = W.make_inputs(wl, seed=4)
    trained = make_layer(wl, inp)
    q = Q4Layer.from_layer(trained, group=64)
    x = inp["x_bf16"].cuda()
    y = q.forward(x).clone()
    few = torch.cat([q.decode(x[i:i + 8].contiguous()).float().clone() for i in range(0, 96, 8)])
    # hidden rows, the experts' outputs and the shared branch's are rounded to bf16 on one
    # side, y on the other
    assert_close("decode", np64(few), np64(y), 2e-2)
    full = trained.forward(x)
    err = float((y - full).norm() / full.norm())
    assert 0.01 < err < 0.3, err                     # 4-bit weights, and close to the layer
    codes = q.matrices["w1"].codes.clone()
    for _ in range(3):
        trained.train_step(x, inp["target"].cuda(), 50.0)
    assert torch.equal(q.matrices["w1"].codes, codes)    # (the router's weights are the layer's own)
    q.requantize(trained)
    assert not torch.equal(q.matrices["w1"].codes, codes)
    y2 = q.forward(x)
    fresh = Q4Layer.from_layer(trained, group=64)
    assert torch.equal(fresh.forward(x), y2)


def test_block_prompt_tokens_graph():
    """Norm and layer together: prompt and tokens, from a captured graph as well."""
    wl = _wl(T=160, D=256, F=128, E=16, k=4)
    inp, ms = _quantized(wl, 8, 32)
    layer = Q4Layer(**_args(wl, inp, ms), max_tokens=160)
    g = torch.Generator("cuda").manual_seed(1)
    gamma = 1 + 0.1 * torch.randn(wl.D, device="cuda", generator=g)
    block = Q4Block(LayerNorm(gamma, None, x_dtype="bf16", z_dtype="bf16"), layer)
    h = torch.randn(160, wl.D, device="cuda", generator=g).bfloat16()
    delta = torch.randn(160, wl.D, device="cuda", generator=g)
    h1, y = block.forward(h, delta)
    assert torch.equal(h1, (h.float() + delta).bfloat16())
    h2, t = block.decode(h[:8].contiguous(), delta[:8].contiguous())
    assert torch.equal(h2, h1[:8])
    assert_close("tokens", np64(t), np64(y[:8]), 2e-2)
    t = t.clone()
    y = y.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hb, db = h.clone(), delta.clone()
    h8, d8 = h[:8].contiguous(), delta[:8].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _, yg = block.forward(hb, db)
        _, tg = block.decode(h8, d8)
    for _ in range(2):
        yg.zero_()
        tg.zero_()
        graph.replay()
        assert torch.equal(yg, y) and torch.equal(tg, t)
    assert layer.status() == 0 and layer.decoder.status() == 0


def test_refused_calls():
    wl = _wl(T=4, D=64, F=32)
    inp, ms = _quantized(wl, 0, 32)
    args = _args(wl, inp, ms)
    layer = Q4Layer(**args, max_tokens=4)
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(4, 64, device="cuda"))
    assert layer.forward(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 64)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(ValueError, match="captured"):
                Q4Layer(**args, max_tokens=4)
            layer.workspace[:1].zero_()


@pytest.mark.parametrize("group,kw", [
    (64, dict(D=16384, F=32, E=256, k=32)), (32, dict(D=32, F=8192, E=256, k=32)),
    (128, dict(D=64, F=4096, E=256, k=32, n_shared=2)), (64, dict(D=16384, F=32, E=32, k=25)),
    (32, dict(D=32, F=8192, E=64, k=32, act="relu", has_bias=True)),
])
def test_decode_widest_rows_beside_the_longest_lists(group, kw):
    """Every layer within the limits is served: rows of the greatest width beside the lists
    of the most tokens."""
    wl = _wl(T=64, **kw)
    inp, ms = _quantized(wl, 9, group)
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=wl.T)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("group,F", [(64, 160), (128, 160), (128, 544)])
@pytest.mark.parametrize("T", [1, 3, 6, 20])
def test_decode_infinite_scale_of_a_short_group(T, group, F):
    """An infinite scale of a group that ends with its inputs gives the infinity of its sum:
    positive hidden activations and weights."""
    wl = _wl(T=T, D=96, F=F, E=8, k=8, act="relu", has_bias=True)
    inp, _ = _quantized(wl, 3, group)
    inp["b1"] = inp["b1"].abs() + 50.0               # every hidden activation is positive
    ms = {n: quantize(inp[n].cuda(), group) for n in ("w1", "w2")}
    last = F // group
    codes = ms["w2"].codes
    codes[:, 5, last * group // 2:] = 0xee           # codes of 14
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=T)
    x = device_x(wl, inp)
    want = d.decode(x).clone()
    ms["w2"].scales[:, last, 5] = float("inf")
    got = d.decode(x)
    rest = [i for i in range(96) if i != 5]
    assert torch.equal(got[:, rest], want[:, rest]) and bool(want.isfinite().all())
    assert bool((got[:, 5] == float("inf")).all())


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("kw", [dict(D=64, F=8224), dict(D=16416, F=32), dict(D=32, F=4128, n_shared=2)])
def test_forward_past_the_few_token_limits(kw, T):
    wl = _wl(T=T, E=8, k=2, **kw)
    inp, ms = _quantized(wl, 6, 128)
    layer = Q4Layer(**_args(wl, inp, ms), max_tokens=T)
    assert layer.decoder is None
    x = device_x(wl, inp)
    y = layer.forward(x)
    assert layer.status() == 0
    want = _forward_want(wl, inp, layer, x, _routing_of(layer, T, wl.k, wl.E))
    assert_close("y", np64(y), want, TOL["bf16"])


def test_from_a_layer_past_the_few_token_limits():
    """A trained layer of wide experts has a 4-bit form as well."""
    wl = _wl(T=40, D=64, F=8224)
    inp = _inputs(wl, 2)
    inp["target"] = torch.zeros(40, 64)
    q = Q4Layer.from_layer(make_layer(wl, inp), group=32)
    x = device_x(wl, inp)
    assert q.decoder is None and q.matrices["w1"].shape == (8, 8224, 64)
    assert bool(q.forward(x).isfinite().all()) and q.status() == 0


@pytest.mark.parametrize("T", [9, 33, 64])
@pytest.mark.parametrize("group,kw", [
    (32, dict(D=64, F=4096, E=8, k=4)), (64, dict(D=96, F=8192, E=8, k=2, act="relu", has_bias=True)),
    (128, dict(D=160, F=4128, E=8, k=4, act="gelu_tanh", has_bias=True)), (64, dict(D=16384, F=64, E=8, k=3)),
    (128, dict(D=64, F=2080, E=16, k=4, n_shared=2)), (32, dict(D=8224, F=96, E=8, k=8, capacity_factor=0.5)),
    (64, dict(D=32, F=5632, E=16, k=4, zipf_skew=1.2, zipf_empty=4)),
    (32, dict(D=64, F=4096, E=32, k=8, score="sigmoid", n_groups=4, topk_groups=2, corr_bias_scale=0.1)),
])
def test_decode_wide_rows(group, kw, T):
    """The form of eight warps: every kind of layer whose rows are wide."""
    wl = _wl(T=T, **kw)
    inp, ms = _quantized(wl, T, group)
    d = MoEDecoder(**_args(wl, inp, ms), max_tokens=T)
    x = device_x(wl, inp)
    y = d.decode(x).clone()
    _check(wl, inp, d, y)
    assert torch.equal(d.decode(x), y)

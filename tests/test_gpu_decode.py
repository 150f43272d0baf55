"""The layer for a few tokens (moe_decode) against the float64 oracle: every
activation, score, type and option of the layer, token counts on both sides of
the kernel's token tiles, rows that end inside its copies, inputs that fit its
shared memory and inputs that do not.

Tolerances.  The kernel's fp32 dot products of K terms add at most K/32 + 10
terms one after another (a lane's share, then a tree); rounding errors of such a
sum have a standard deviation of at most 2^-25 sqrt(K/32 + 10) of its largest
partial sum, and 16 of those cover every output of a test.  Two products in a
row and the activation between them (slope at most 1.2, times a factor of the
same size for SwiGLU) are covered by a factor 4.  The result is rounded once to
the layer's type: half a step, 2^-8 of the value for bf16.
"""

import dataclasses
import math

import numpy as np
import pytest
import torch

import workloads as W
from oracle import moe_oracle as O
from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder
from tests.moe_cases import (device_x, make_layer, np64, oracle_config, oracle_inputs,
                             validated_routing)

pytestmark = pytest.mark.gpu


def _f32_tol(D, F):
    return 4 * 16 * 2.0 ** -25 * math.sqrt(max(D, F) / 32 + 10)


def _wl(**kw):
    base = dict(name="t", T=1, D=64, F=32, E=8, k=2, act="swiglu", score="softmax", n_groups=1,
                topk_groups=1, has_bias=False, dtype="bf16", aux_alpha=0.0, lr=0.1)
    base.update(kw)
    return W.Workload(**base)


def _inputs(wl, seed):
    inp = W.make_inputs(wl, seed=seed, with_target=False)
    inp["target"] = None
    if wl.has_bias:     # the training recipe starts them at zero
        g = torch.Generator().manual_seed(seed + 11)
        inp["b1"] = 0.3 * torch.randn(wl.E, wl.F, generator=g)
        inp["b2"] = 0.3 * torch.randn(wl.E, wl.D, generator=g)
    return inp


def _decoder(wl, inp, group_score="top2_sum", max_tokens=None):
    lp = "_bf16" if wl.dtype == "bf16" else ""
    c = lambda t: None if t is None else t.cuda().contiguous()  # noqa: E731
    return MoEDecoder(c(inp["w_gate"]), c(inp["w1" + lp]), c(inp["w2" + lp]),
                      w3=c(inp["w3" + lp]) if inp["w3"] is not None else None, b1=c(inp["b1"]),
                      b2=c(inp["b2"]), k=wl.k, act=wl.act, score=wl.score, n_groups=wl.n_groups,
                      topk_groups=wl.topk_groups, group_score=group_score,
                      logit_bias=c(inp["logit_bias"]), corr_bias=c(inp["corr_bias"]),
                      n_shared=wl.n_shared, ws1=c(inp.get("ws1" + lp)),
                      ws3=c(inp.get("ws3" + lp)), ws2=c(inp.get("ws2" + lp)),
                      capacity_factor=wl.capacity_factor, max_tokens=max_tokens or max(wl.T, 1))


def _check(wl, inp, d, y, group_score="top2_sum"):
    cfg = oracle_config(wl, group_score)
    w, _, x, _ = oracle_inputs(wl, inp)
    idx_gpu = d.idx.cpu().numpy()
    scores = O.router_scores(cfg, O.router_logits(x, w["w_gate"], w["logit_bias"]))
    idx = validated_routing(cfg, scores, idx_gpu, corr_bias=w["corr_bias"])
    st = O.forward(cfg, w, x, idx)
    tol = _f32_tol(wl.D, wl.F * max(1, wl.n_shared))
    # a gate's error: the logits' (times their size), plus the exponential and a division
    logit = np.abs(st["logits"][np.isfinite(st["logits"])]).max() + 1
    assert np.abs(d.gate.cpu().numpy() - st["gate"]).max() <= tol * logit
    got, want = np64(y), st["y"]
    half = 2.0 ** -8 if wl.dtype == "bf16" else 2.0 ** -24
    # the activations' sizes, not those of their sum, scale the fp32 part
    amp = max(np.abs(st["ye"]).max() if st["ye"].size else 0.0, np.abs(want).max())
    bad = np.abs(got - want) > half * np.abs(want) + tol * logit * amp
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.abs(got - want).max():.3e}"
    assert d.status() == 0


TOKENS = [1, 2, 3, 5, 7, 8, 9, 16, 17, 33, 64]
CASES = {
    "relu_bias_f32": dict(act="relu", has_bias=True, dtype="f32", D=32, F=64, E=4),
    "gelu_bias_f32": dict(act="gelu_tanh", has_bias=True, dtype="f32", D=200, F=328),
    "gelu_nobias_bf16": dict(act="gelu_tanh", D=512, F=264, E=16, k=3),
    "relu_bias_bf16": dict(act="relu", has_bias=True, D=264, F=520, k=4),
    "swiglu_f32": dict(dtype="f32", D=136, F=72, E=20, k=5),
    "swiglu_bf16": dict(D=1024, F=704, E=16, k=4),
    "grouped_sigmoid": dict(score="sigmoid", n_groups=8, topk_groups=4, E=64, k=6, D=256, F=88),
    "corrected": dict(score="sigmoid", n_groups=4, topk_groups=2, E=32, k=4, corr_bias_scale=0.1),
    "shared": dict(n_shared=2, E=16, k=2, D=328, F=200),
    "skewed_empty": dict(E=16, k=4, zipf_skew=1.2, zipf_empty=4, D=128, F=136),
    "smallest": dict(D=8, F=8, E=8, k=1),
    "every_expert": dict(E=8, k=8, D=72, F=40),
}


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("name", sorted(CASES))
def test_decode(name, T):
    wl = _wl(T=T, **CASES[name])
    inp = _inputs(wl, seed=T)
    d = _decoder(wl, inp)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("kw", [
    dict(T=33, D=4096, F=64, E=8),                      # tokens past the shared memory
    dict(T=48, D=512, F=704, E=8, k=8),                 # hidden activations past it
    dict(T=40, D=4096, F=1024, E=8, k=4, n_shared=1),   # both, and several row batches
    dict(T=24, D=2048, F=512, E=8, dtype="f32"),
    dict(T=64, D=32, F=16, E=256, k=32),                # the most routed rows
    dict(T=64, D=64, F=16, E=256, k=32, dtype="f32", n_groups=32, topk_groups=32,
         score="sigmoid"),
    dict(T=1, D=8, F=2048, E=8), dict(T=1, D=8192, F=8, E=8),
    dict(T=3, D=16384, F=24, E=8, n_shared=1),
    # the widest rows the kernel takes, beside the longest lists
    dict(T=64, D=16384, F=16, E=256, k=32), dict(T=64, D=16, F=8192, E=16, k=16),
    dict(T=9, D=16, F=4096, E=8, n_shared=2),
    dict(T=33, D=8192, F=16, E=8, k=3, dtype="f32"), dict(T=5, D=16, F=8192, E=8, dtype="f32"),
    dict(T=64, D=7168, F=256, E=8, k=2),                # tiles of an odd number of tokens
], ids=lambda kw: "_".join(f"{k}{v}" for k, v in kw.items()))
def test_decode_extremes(kw):
    wl = _wl(**kw)
    inp = _inputs(wl, seed=3)
    d = _decoder(wl, inp)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("name,T", [("tiny", 64), ("grouped", 1), ("grouped_cb", 12),
                                    ("grouped_shared", 5), ("dense_f32_cap", 31),
                                    ("dense_bf16", 20)])
def test_decode_configured_layers(name, T):
    wl = W.WORKLOADS[name].with_tokens(T)
    inp = _inputs(wl, seed=1)
    d = _decoder(wl, inp)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


@pytest.mark.parametrize("cf", [0.1, 0.5, 1.0, 4.0])
def test_decode_capacity(cf):
    wl = _wl(T=37, E=8, k=3, capacity_factor=cf, act="relu", has_bias=True, dtype="f32")
    inp = _inputs(wl, seed=2)
    d = _decoder(wl, inp)
    _check(wl, inp, d, d.decode(device_x(wl, inp)))


def test_decode_group_max_and_ties():
    """Equal scores go to the smaller id, in groups and out of them."""
    for groups, top in ((1, 1), (4, 2)):
        wl = _wl(T=6, E=16, k=3, n_groups=groups, topk_groups=top)
        inp = _inputs(wl, seed=4)
        inp["w_gate"] = torch.zeros_like(inp["w_gate"])
        d = _decoder(wl, inp, group_score="max")
        d.decode(device_x(wl, inp))
        assert d.idx.tolist() == [[0, 1, 2]] * 6
        assert torch.allclose(d.gate, torch.full_like(d.gate, 1 / 3))
    wl = _wl(T=9, E=16, k=3, n_groups=4, topk_groups=2, score="sigmoid")
    inp = _inputs(wl, seed=5)
    d = _decoder(wl, inp, group_score="max")
    _check(wl, inp, d, d.decode(device_x(wl, inp)), group_score="max")


def test_decode_matches_the_training_forward():
    """moe_forward on the same tokens: the same routing (up to near-ties of its
    own tensor-core logits) and the same y up to its bf16 hidden rows."""
    wl = dataclasses.replace(W.WORKLOADS["grouped"], T=48)
    inp = _inputs(wl, seed=6)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    y = d.decode(x)
    layer = make_layer(wl, inp)
    want = layer.forward(x)
    same = (d.idx == layer.routing()["idx"]).all(1)
    assert int(same.sum()) >= 46
    # three bf16 roundings (hidden rows, Y_e, y), each half a step of its value
    err = (y.float() - want)[same].abs().max() / want.abs().max()
    assert err <= 3 * 2.0 ** -8


def test_decode_a_bad_token_stays_alone():
    wl = _wl(T=11, D=264, F=136, E=16, k=4)
    inp = _inputs(wl, seed=7)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    clean = d.decode(x).clone()
    x[4, 100] = float("nan")
    x[9, 0] = float("inf")
    y = d.decode(x)
    assert torch.isnan(y[4]).all()
    for t in set(range(11)) - {4, 9}:
        assert torch.equal(y[t], clean[t]), t
    assert d.status() == 0


@pytest.mark.parametrize("act,dtype", [("relu", "f32"), ("relu", "bf16"), ("gelu_tanh", "f32")])
def test_decode_a_nan_passes_the_activation(act, dtype):
    """A NaN hidden value reaches y (ReLU does not turn it into a zero), in the
    tokens of its expert only."""
    wl = _wl(T=12, D=64, F=32, E=8, k=1, act=act, dtype=dtype, has_bias=True)
    inp = _inputs(wl, seed=12)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    clean = d.decode(x).clone()
    e = int(d.idx[0, 0])
    inp["b1"][e, 5] = float("nan")
    d = _decoder(wl, inp)
    y = d.decode(x)
    hit = d.idx[:, 0] == e
    assert torch.isnan(y[hit]).all()
    assert torch.equal(y[~hit], clean[~hit])


def test_decode_token_counts_share_a_decoder():
    wl = _wl(T=64, D=328, F=72, E=16, k=3, n_shared=1)
    inp = _inputs(wl, seed=8)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    whole = d.decode(x).clone()
    routing = d.idx.clone()
    for T in (1, 40, 3, 64, 8, 17):
        y = d.decode(x[:T].contiguous())
        assert y.shape == (T, 328) and d.idx.shape == (T, 3)
        # the order of a token's sums goes with the call's split of the work, its
        # routing does not; two roundings of nearly equal values: a step at most
        want = whole[:T].float()
        tol = 2.0 ** -7 * want.abs() + _f32_tol(328, 72) * want.abs().max()
        assert ((y.float() - want).abs() <= tol).all()
        assert torch.equal(d.idx, routing[:T])
        assert torch.equal(y, d.decode(x[:T].contiguous(), y=torch.empty_like(y)))
    assert d.decode(x[:0]).shape == (0, 328)
    assert d.status() == 0


def test_decode_on_a_side_stream_and_in_a_graph():
    wl = _wl(T=6, D=256, F=136, E=16, k=3)
    inp = _inputs(wl, seed=9)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    want = d.decode(x).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = d.decode(x).clone()
    s.synchronize()
    assert torch.equal(y, want)
    out, x2 = torch.zeros_like(want), x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        d.decode(x2, y=out)
        d.decode(out, y=x2)
        d.decode(x2, y=out)
    graph.replay()
    torch.cuda.synchronize()
    a = d.decode(x).clone()
    b = d.decode(a).clone()
    assert torch.equal(d.decode(b), out)
    graph.replay()
    torch.cuda.synchronize()
    assert d.status() == 0


def test_decode_refuses_a_workspace_without_init():
    wl = _wl(T=2)
    inp = _inputs(wl, seed=10)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    want = d.decode(x).clone()
    d.workspace.zero_()
    d.decode(x, y=torch.zeros_like(want))
    assert d.status() == B.MOE_ERR_INVALID_ARG
    d.reset()
    assert torch.equal(d.decode(x), want) and d.status() == 0


def test_decode_weights_past_32_bit_offsets():
    """More than 2^31 values a tensor: the last experts' rows are read."""
    E, F, D = 72, 4096, 8192
    g = torch.Generator("cuda").manual_seed(1)
    mk = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(  # noqa: E731
        0, s[-1] ** -0.5, generator=g)
    w1, w2 = mk(E, F, D), mk(E, D, F)
    assert w1.numel() > 1 << 31
    w_gate = torch.zeros(E, D, device="cuda")
    lb = torch.zeros(E, device="cuda")
    lb[E - 2:] = 30.0
    d = MoEDecoder(w_gate, w1, w2, k=2, act="relu", logit_bias=lb, max_tokens=2)
    x = torch.randn(2, D, device="cuda", generator=g).bfloat16()
    y = d.decode(x)
    assert d.idx.tolist() == [[E - 2, E - 1]] * 2
    want = 0
    for e in (E - 2, E - 1):
        want = want + 0.5 * (x.double() @ w1[e].double().t()).clamp(min=0) @ w2[e].double().t()
    tol = 2.0 ** -8 * want.abs() + _f32_tol(D, F) * want.abs().max()
    assert ((y.double() - want).abs() <= tol).all()


def test_largest_hidden_values():
    """bf16 layers: a hidden value beyond the largest bf16 stays itself, and an
    infinite one gives infinities, not NaN."""
    E, F, D = 8, 32, 64
    w1, w2 = torch.zeros(E, F, D), torch.zeros(E, D, F)
    x = torch.zeros(2, D)
    x[0, 0], x[0, 1], x[1, 2] = 2.0 ** 127, 2.0 ** 119, 2.0 ** 127
    w1[0, 0, 0], w1[0, 0, 1], w1[0, 1, 2] = 1.9921875, 1.5, 4.0
    w2[0, :, 0], w2[0, 0::2, 1], w2[0, 1::2, 1] = 2.0 ** -10, 1.0, -1.0
    lb = torch.zeros(E, device="cuda")
    lb[0] = 200.0                                     # expert 0 with gate 1
    c = lambda t: t.bfloat16().cuda()  # noqa: E731
    d = MoEDecoder(torch.zeros(E, D, device="cuda"), c(w1), c(w2), k=1, act="relu", logit_bias=lb,
                   max_tokens=2)
    y = d.decode(c(x)).double().cpu()
    h = 2.0 ** 127 * 1.9921875 + 1.5 * 2.0 ** 119     # fits fp32, rounds past bf16
    assert ((y[0] - 2.0 ** -10 * h).abs() <= 2.0 ** -8 * 2.0 ** -10 * h).all()
    assert (y[1, 0::2] == math.inf).all() and (y[1, 1::2] == -math.inf).all()


@pytest.mark.parametrize("F", [32, 2048])          # one warp an item, and several
def test_infinite_down_weights(F):
    """bf16 layers: an infinite W2 value times a hidden value is an infinity of its
    sign, and so is a product past fp32's range, whatever the second part of the
    hidden value is (zero, of the same sign, of the other sign)."""
    E, D = 8, 64
    w1, w2 = torch.zeros(E, F, D), torch.zeros(E, D, F)
    h = [2.0, 1 + 2.0 ** -9, 1 + 1.5 * 2.0 ** -8, 2048 * (1 + 1.5 * 2.0 ** -8)]
    x = torch.zeros(4, D)
    for t, v in enumerate(h):                         # token t: hidden value 0 of expert 0 is h[t]
        first = float(torch.tensor(v).bfloat16())
        x[t, 2 * t], x[t, 2 * t + 1] = first, v - first
        w1[0, 0, 2 * t] = w1[0, 0, 2 * t + 1] = 1.0
    w2[0, 1, 0], w2[0, 2, 0], w2[0, 3, 0], w2[0, 4, 0] = math.inf, -math.inf, 3e38, -3e38
    w2[0, 5, 0] = 1.0
    lb = torch.zeros(E, device="cuda")
    lb[0] = 200.0                                     # expert 0 with gate 1
    c = lambda t: t.bfloat16().cuda()  # noqa: E731
    d = MoEDecoder(torch.zeros(E, D, device="cuda"), c(w1), c(w2), k=1, act="relu", logit_bias=lb,
                   max_tokens=4)
    for T in (4, 1):
        y = d.decode(c(x[4 - T:])).double().cpu()
        assert (y[:, 1] == math.inf).all() and (y[:, 2] == -math.inf).all()
        assert y[-1, 3] == math.inf and y[-1, 4] == -math.inf
        want = torch.tensor(h[4 - T:], dtype=torch.float64)
        assert ((y[:, 5] - want).abs() <= 2.0 ** -8 * want).all()
        assert not y[:, 0].any() and not y[:, 6:].any()
    assert d.status() == 0


def test_a_decoder_is_not_made_in_a_capture():
    """Its workspace would be cleared by the graph's replays only."""
    wl = _wl(T=2)
    inp = _inputs(wl, seed=13)
    x = device_x(wl, inp)
    d = _decoder(wl, inp)
    want = d.decode(x).clone()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    weights = [inp[n].cuda() for n in ("w_gate", "w1_bf16", "w2_bf16", "w3_bf16")]
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captur"):
            MoEDecoder(weights[0], weights[1], weights[2], w3=weights[3], k=wl.k, act=wl.act)
        d.decode(x, y=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_an_expired_grid_barrier_ends_in_order(which):
    """A barrier's counter that starts one low never fills: every block's wait runs
    out (2 s), the call ends, the status says so, and a reset restores the decoder."""
    wl = _wl(T=6, D=256, F=136, E=16, k=3, n_shared=1)
    inp = _inputs(wl, seed=14)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    want = d.decode(x).clone()
    assert d.status() == 0
    counters = d.workspace[:256].view(torch.int32)
    assert counters[32:35].tolist() == [0, 0, 0]     # ready for the next call
    counters[32 + which] = -1
    d.decode(x)
    assert d.status() == B.MOE_ERR_TIMEOUT
    assert counters[32:35].tolist() == [0, 0, 0]
    d.reset()
    assert torch.equal(d.decode(x), want)
    assert d.status() == 0


def test_direct_bindings():
    """The binding's functions, as a program without the class calls them."""
    wl = _wl(T=5, D=136, F=72, E=16, k=3)
    inp = _inputs(wl, seed=15)
    d = _decoder(wl, inp)
    x = device_x(wl, inp)
    want = d.decode(x)
    w = [inp[n].cuda() for n in ("w_gate", "w1_bf16", "w2_bf16", "w3_bf16")]
    cfg = B.make_config(5, 136, 72, 16, 3, act="swiglu", score=wl.score, dtype="bf16",
                        has_bias=False)
    weights = B.make_weights(w[0], w[1], w[2], w3=w[3])
    ws = torch.empty(B.moe_decode_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    y, idx, gate = torch.empty_like(x), torch.empty_like(d.idx), torch.empty_like(d.gate)
    B.moe_decode_init(cfg, ws)
    B.moe_decode(cfg, weights, x, y, ws, idx=idx, gate=gate)
    assert B.moe_last_launch_count() == 1
    assert torch.equal(y, want) and torch.equal(idx, d.idx) and torch.equal(gate, d.gate)
    y.zero_()
    B.moe_decode(cfg, weights, x, y, ws)              # the routing is optional
    assert torch.equal(y, want) and B.moe_decode_status(cfg, ws) == 0

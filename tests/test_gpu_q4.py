"""4-bit expert weights on the GPU against plain float64 arithmetic: quantising and
reading back (exact), and the grouped product over segment lengths on both sides of
the kernels' row tiles, ragged and empty segments, short last groups, every activation.

Tolerances: tests/q4_cases.py derives the bound of a product's fp32 sums; the result is
rounded once to bf16 (half a step, 2^-8 of the value)."""

import numpy as np
import pytest
import torch

from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.q4 import Q4Matrix, Q4Product, quantize
from tests import q4_cases as C

pytestmark = pytest.mark.gpu


# ---- quantising and reading back

def _hard_weights(rng, E, N, K, group, dtype):
    """Random weights with what is hard among them: groups of zeros, values on and next to
    the border of two codes, tiny and huge groups."""
    w = rng.normal(0, K ** -0.5, (E, N, K))
    w[:, 0, :] = 0.0
    w[:, 1, :] *= 1e-41                          # below the normal numbers of fp32
    w[:, 2, :] *= 1e34
    w[:, 3, :] *= 2.0 ** -64
    s = 1.25 * 2.0 ** rng.integers(-8, 8)        # a scale of five bits: 7 s is the largest
    border = rng.integers(-7, 7, (E, K)) + 0.5
    w[:, 4, :] = border * s
    w[:, 4, ::group] = 7 * s
    w = torch.from_numpy(w).to(dtype)
    if dtype is torch.float32:                   # one last place on either side of a border
        step = torch.tensor(rng.choice([-1, 1], (E, K)))
        v = w[:, 4].clone()
        side = torch.nextafter(v, torch.where(step > 0, torch.inf, -torch.inf).float())
        side[:, ::group] = v[:, ::group]
        w[:, 5] = side
    return w


@pytest.mark.parametrize("group", B.Q4_GROUPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 8, 32), (3, 16, 96), (2, 40, 704), (5, 8, 256), (1, 24, 1056),
                                   (2, 72, 512)])
def test_quantize(shape, dtype, group):
    E, N, K = shape
    w = _hard_weights(np.random.default_rng(N + K), E, N, K, group, dtype)
    codes, scales = C.quantize(w.double().numpy(), group)
    q = quantize(w.cuda(), group)
    assert np.array_equal(q.scales.double().cpu().numpy(), scales)
    assert np.array_equal(C.unpack(q.codes.cpu().numpy()), codes)
    want = C.weights(codes, scales, group)
    for out_type in (torch.bfloat16, torch.float32):
        got = q.dequantize(out_type)
        assert got.dtype is out_type
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert np.abs(codes - 8).max() == 7


def test_quantize_not_finite():
    w = torch.randn(1, 16, 128)
    w[0, 3, 5], w[0, 4, 70], w[0, 5, 127] = float("nan"), float("inf"), -float("inf")
    q = quantize(w.cuda(), 64)
    s = q.scales.cpu()[0]
    bad = torch.zeros(2, 16, dtype=torch.bool)
    bad[0, 3] = bad[1, 4] = bad[1, 5] = True
    assert torch.equal(s.isnan(), bad)
    v = q.dequantize().cpu()[0]
    assert torch.equal(v.isnan(), bad.t().repeat_interleave(64, 1))


@pytest.mark.parametrize("five", [True, False])
def test_dequantize_every_code(five):
    rng = np.random.default_rng(3)
    codes, scales = C.random_matrix(rng, 3, 40, 160, 64, five)
    m = C.device_matrix(codes, scales, 64)
    assert np.array_equal(m.dequantize().double().cpu().numpy(), C.weights(codes, scales, 64))


@pytest.mark.parametrize("shape", [(1, 8, 32), (3, 40, 352), (2, 16, 8192)])
def test_pack_stays_in_its_tensors(shape):
    """Nothing is written behind codes, scales or weights."""
    E, N, K = shape
    G = -(-K // 64)
    codes = torch.full((E * N * K // 2 + 64,), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((E * G * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    q = Q4Matrix(codes[:-64].view(E, N, K // 2), scales[:-64].view(E, G, N), 64)
    quantize(torch.randn(E, N, K, device="cuda"), 64, out=q)
    assert (codes[-64:] == 7).all() and (scales[-64:] == 7).all() and (codes[:-64] != 7).any()
    for dt in (torch.bfloat16, torch.float32):
        w = torch.full((E * N * K + 64,), 7.0, dtype=dt, device="cuda")
        q.dequantize(out=w[:-64].view(E, N, K))
        assert (w[-64:] == 7).all()


def test_quantize_in_place_and_2d():
    w = torch.randn(24, 96, device="cuda")
    q = quantize(w, 32)
    assert q.shape == (1, 24, 96)
    first = C.unpack(q.codes.cpu().numpy()).astype(int)
    assert quantize(-w, 32, out=q) is q
    assert np.array_equal(C.unpack(q.codes.cpu().numpy()), 16 - first)


# ---- the grouped product

def _product_case(seed, counts, N, K, group, act, bias, five=True, before=0, behind=0):
    rng = np.random.default_rng(seed)
    E = len(counts)
    m = C.random_matrix(rng, E, N, K, group, five)
    m3 = C.random_matrix(rng, E, N, K, group, five) if act == "swiglu" else None
    b = rng.normal(0, 0.5, (E, N)).astype(np.float32) if bias else None
    R = before + sum(counts) + behind
    x = C.bf16(rng.normal(0, 1, (R, K)))
    offsets = before + np.concatenate([[0], np.cumsum(counts)])
    return dict(m=m, m3=m3, b=b, x=x, offsets=offsets, R=R, N=N, group=group, act=act)


def _device(c):
    p = Q4Product(C.device_matrix(*c["m"], c["group"]),
                  None if c["m3"] is None else C.device_matrix(*c["m3"], c["group"]),
                  bias=None if c["b"] is None else torch.from_numpy(c["b"]).cuda(), act=c["act"])
    return (p, torch.from_numpy(c["x"]).bfloat16().cuda(),
            torch.from_numpy(c["offsets"]).int().cuda())


def _check(c, got, fill=None):
    got = got.double().cpu().numpy()
    w = C.weights(*c["m"], c["group"])
    w3 = C.weights(*c["m3"], c["group"]) if c["m3"] is not None else None
    used = np.zeros(c["R"], bool)
    for e, (lo, hi) in enumerate(zip(c["offsets"][:-1], c["offsets"][1:])):
        if lo == hi:
            continue
        used[lo:hi] = True
        y, err = C.product_row_block(c["act"], c["x"][lo:hi], w[e], None if w3 is None else w3[e],
                                     None if c["b"] is None else c["b"][e].astype(np.float64))
        bad = np.abs(got[lo:hi] - y) > C.BF16_HALF * np.abs(y) + err * (1 + C.BF16_HALF)
        assert not bad.any(), (e, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                               float(np.abs(got[lo:hi] - y).max()))
    if fill is not None:
        assert (got[~used] == fill).all()


COUNTS = {
    "one": [1], "few": [3, 0, 2, 1], "eights": [7, 8, 9], "sixteens": [15, 16, 17, 0, 33],
    "tile": [63, 64, 65], "tiles": [127, 128, 129, 1], "wide": [255, 0, 256, 257], "long": [600, 5, 0, 301],
    "empty": [0, 0, 0], "last": [0, 0, 40],
}
SHAPES = [(8, 32, 32), (64, 64, 64), (136, 96, 32), (200, 480, 64), (256, 704, 128), (72, 1056, 64),
          (520, 160, 128)]


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act,bias", [("none", False), ("gelu_tanh", True), ("relu", True), ("swiglu", False)])
def test_product(act, bias, shape, name):
    N, K, group = shape
    c = _product_case(N + K + len(name), COUNTS[name], N, K, group, act, bias, before=2, behind=3)
    p, x, off = _device(c)
    out = torch.full((c["R"], N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert p.forward(x, off, out) is out
    _check(c, out, fill=7.0)
    assert p.status() == 0


@pytest.mark.parametrize("counts,N,K,group,act", [
    ([1], 4096, 2048, 64, "none"), ([2], 2048, 4096, 128, "swiglu"), ([1], 64, 8192, 32, "none"),
    ([24, 0, 5], 1408, 2048, 128, "swiglu"), ([300], 1000, 480, 64, "gelu_tanh"),
    ([2, 1, 0, 3] * 16, 704, 1024, 64, "swiglu"), ([1] * 256, 64, 64, 32, "none"),
    ([700, 20, 0, 90], 512, 4096, 32, "none"), ([1], 16, 65536, 128, "none"), ([40], 16, 65536, 64, "none"),
])
def test_product_sizes(counts, N, K, group, act):
    c = _product_case(5, counts, N, K, group, act, False)
    p, x, off = _device(c)
    _check(c, p.forward(x, off))
    assert p.status() == 0


# more rows than the few-row kernel takes: segments around the row tiles of the other
MANY = [4100, 1, 0, 15, 16, 17, 33, 64, 65, 96, 97, 127, 128, 129, 159, 160, 161, 0, 320, 321, 480, 5]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act,bias", [("none", False), ("gelu_tanh", True), ("relu", True), ("swiglu", False)])
def test_product_many_rows(act, bias, shape):
    N, K, group = shape
    c = _product_case(N + 2 * K, MANY, N, K, group, act, bias, before=2, behind=3)
    p, x, off = _device(c)
    out = torch.full((c["R"], N), 7.0, dtype=torch.bfloat16, device="cuda")
    p.forward(x, off, out)
    _check(c, out, fill=7.0)
    assert p.status() == 0


@pytest.mark.parametrize("counts,N,K,group,act", [
    ([0, 4096], 8, 32, 32, "none"), ([4096, 1], 8, 32, 32, "none"), ([4097], 8, 32, 32, "swiglu"),
    ([17] * 256, 16, 96, 64, "none"), ([0] * 255 + [5000], 40, 64, 32, "relu"),
    ([4000, 600], 136, 8192, 128, "none"), ([5000], 1000, 32, 32, "swiglu"), ([100] * 64, 704, 1024, 64, "swiglu"),
])
def test_product_many_rows_sizes(counts, N, K, group, act):
    c = _product_case(7, counts, N, K, group, act, act == "relu")
    p, x, off = _device(c)
    _check(c, p.forward(x, off))
    assert p.status() == 0


@pytest.mark.parametrize("counts", [[4], [40, 90], [300], [3000, 1200]])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_scales_of_eight_bits(counts, act):
    c = _product_case(9, counts, 72, 320, 32, act, False, five=False)
    p, x, off = _device(c)
    _check(c, p.forward(x, off))


@pytest.mark.parametrize("counts,scale", [([4], 1e-3), ([4], 2.0 ** -119), ([4], 2.0 ** 20), ([40, 90], 8.0),
                                          ([3000, 1200], 2.0 ** -122), ([3000, 1200], 2.0 ** 30)])
def test_product_scales_of_any_size(counts, scale):
    """Scales on both sides of the range of the kernels' short way to widen a code, in one
    matrix: some groups are `scale` times the others, which are exact zeros in places."""
    c = _product_case(21, counts, 72, 320, 32, "none", False)
    codes, s = c["m"]
    s = s.copy()
    s[:, ::3] *= scale
    s[:, 1, ::5] = 0.0
    c["m"] = (codes, C.bf16(s))
    p, x, off = _device(c)
    _check(c, p.forward(x, off))


@pytest.mark.parametrize("counts", [[4], [40, 90], [3000, 1200]])
@pytest.mark.parametrize("low,high", [(-133, -126), (-130, -110), (-121, -116)])
def test_product_smallest_scales(counts, low, high):
    """Weights down to the least bf16 number.  The kernels round a weight once, to a
    multiple of 2^-125 where it is below 2^-118 (half a step: 2^-126), the plain form to a
    multiple of 2^-133 or 8 bits (half a step below 2^-118: 2^-127)."""
    c = _product_case(23, counts, 72, 320, 32, "none", False)
    codes, s = c["m"]
    rng = np.random.default_rng(24)
    c["m"] = (codes, C.bf16(np.ldexp(rng.uniform(1, 2, s.shape), rng.integers(low, high, s.shape))))
    c["x"] = C.bf16(np.ldexp(c["x"], 60))
    p, x, off = _device(c)
    got = p.forward(x, off).double().cpu().numpy()
    w = C.weights(*c["m"], 32)
    for e, (lo, hi) in enumerate(zip(c["offsets"][:-1], c["offsets"][1:])):
        y, err = C.product_row_block("none", c["x"][lo:hi], w[e])
        err = err + (2.0 ** -126 + 2.0 ** -127) * np.abs(c["x"][lo:hi]).sum(1, keepdims=True)
        assert (np.abs(got[lo:hi] - y) <= C.BF16_HALF * np.abs(y) + err * (1 + C.BF16_HALF)).all()
    assert p.status() == 0


@pytest.mark.parametrize("counts", [[3, 4], [20, 50], [150, 150], [200, 4000]])
def test_rows_do_not_mix(counts):
    """A row of NaN and one of infinities stay in their rows, a NaN and an infinite scale
    in their outputs; rows outside of the segments are not looked at."""
    c = _product_case(11, counts, 64, 160, 32, "none", False, before=3, behind=5)
    n0, n1 = counts
    x, off = c["x"].copy(), c["offsets"]
    x[:3] = np.nan
    x[-5:] = np.inf
    x[off[0] + 1] = np.nan
    x[off[1] + 2] = np.inf
    clean = [r for r in range(off[0], off[2]) if r not in (off[0] + 1, off[1] + 2)]
    p, _, d_off = _device(c)
    got = p.forward(torch.from_numpy(x).bfloat16().cuda(), d_off).double().cpu().numpy()
    want = p.forward(torch.from_numpy(c["x"]).bfloat16().cuda(), d_off).double().cpu().numpy()
    assert np.array_equal(got[clean], want[clean])
    assert np.isnan(got[off[0] + 1]).all() and not np.isfinite(got[off[1] + 2]).any()
    # scales: output 5 of expert 0 (its last group), output 9 of expert 1
    codes, scales = c["m"][0].copy(), c["m"][1].copy()
    codes[codes == 8] = 9
    scales[0, -1, 5], scales[1, 0, 9] = np.nan, np.inf
    p2 = Q4Product(C.device_matrix(codes, scales, 32))
    got = p2.forward(torch.from_numpy(c["x"]).bfloat16().cuda(), d_off).double().cpu().numpy()
    bad = ~np.isfinite(got[off[0]:off[2]])
    want_bad = np.zeros_like(bad)
    want_bad[:n0, 5] = want_bad[n0:, 9] = True
    assert np.array_equal(bad, want_bad)


def test_offsets_are_clamped():
    """Offsets that decrease, are negative or run past the rows select the rows that the
    clamped sequence has; nothing behind the output is written."""
    c = _product_case(13, [10, 10, 10, 10], 64, 64, 32, "none", False)
    p, x, _ = _device(c)
    for off in ([-5, 10, 4, 30, 40], [0, 100, 20, 30, 1 << 30], [8, 3, 12, 12, 40],
                [-(1 << 31), -1, 7, 7, 50]):
        fixed, prev = [], 0
        for v in off:
            prev = max(prev, min(max(v, prev), 40))
            fixed.append(prev)
        guard = torch.full((60, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        p.forward(x, torch.tensor(off, dtype=torch.int32, device="cuda"), guard[:40])
        assert (guard[40:] == 3).all()
        _check(dict(c, offsets=np.array(fixed)), guard[:40], fill=3.0)


def test_offsets_are_clamped_many_rows():
    c = _product_case(14, [2000, 1000, 0, 1500], 64, 64, 32, "none", False)
    p, x, _ = _device(c)
    for off in ([-5, 10, 4, 30, 4500], [0, 100000, 20, 30, 1 << 30], [8, 3, 12, 4200, 4100]):
        fixed, prev = [], 0
        for v in off:
            prev = max(prev, min(max(v, prev), 4500))
            fixed.append(prev)
        guard = torch.full((4700, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        p.forward(x, torch.tensor(off, dtype=torch.int32, device="cuda"), guard[:4500])
        assert (guard[4500:] == 3).all()
        _check(dict(c, offsets=np.array(fixed)), guard[:4500], fill=3.0)


def test_waits_expire():
    """With its loads withheld the product for many rows ends by itself, says so and writes
    nothing; the next call is not affected."""
    c = _product_case(2, [300, 200], 264, 320, 64, "none", False)
    p, x, off = _device(c)
    cfg = B.moe_q4_product_config(500, 2, 264, 320, 64, B.MOE_Q4_ACT_NONE)
    out = torch.full((500, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    m = C.device_matrix(*c["m"], 64)
    B.moe_q4_selftest_wait_timeout(cfg, off, x, m.c_matrix(), out, status, 20_000_000)
    torch.cuda.synchronize()
    assert status[0] == B.MOE_ERR_TIMEOUT and (out == 7).all()
    _check(c, p.forward(x, off))
    assert p.status() == 0


def test_no_rows():
    c = _product_case(1, [0, 0], 64, 64, 32, "none", False)
    p, _, off = _device(c)
    assert p.forward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), off).shape == (0, 64)


@pytest.mark.parametrize("counts", [[3, 4], [100, 180], [4000, 300]])
def test_streams_and_graphs(counts):
    """The same bits on another stream, from a captured graph, from two streams at once."""
    c = _product_case(17, counts, 264, 320, 64, "swiglu", False)
    p, x, off = _device(c)
    want = p.forward(x, off)
    _check(c, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [p.forward(x, off) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph, buf = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = p.forward(buf, off)
    for k in (1.0, 2.0):
        buf.copy_(x * k)
        graph.replay()
        assert torch.equal(out, p.forward(buf, off))
    assert p.status() == 0


@pytest.mark.parametrize("counts", [[1, 2], [3, 4], [20, 50], [200, 4000]])
@pytest.mark.parametrize("K,group", [(160, 64), (160, 128), (544, 128), (96, 64)])
def test_infinite_scale_of_a_short_group(counts, K, group):
    """An infinite scale of a group that ends with its inputs gives the infinity of its sum:
    positive rows and weights.  The other outputs do not see it."""
    c = _product_case(19, counts, 72, K, group, "none", False)
    last = K // group
    codes, scales = c["m"][0].copy(), c["m"][1].copy()
    codes[:, 5, last * group:] = np.maximum(codes[:, 5, last * group:], 9)
    c["x"] = np.abs(c["x"]) + 2.0 ** -8
    c["x"] = C.bf16(c["x"])
    c["m"] = codes, scales
    p, x, off = _device(c)
    want = p.forward(x, off)
    _check(c, want)
    scales = scales.copy()
    scales[:, last, 5] = np.inf
    got = Q4Product(C.device_matrix(codes, scales, group)).forward(x, off)
    rest = [i for i in range(72) if i != 5]
    assert torch.equal(got[:, rest], want[:, rest])
    assert bool((got[:, 5] == float("inf")).all())


@pytest.mark.parametrize("rows", [40, 777, 5000])
def test_product_gelu_of_negative_inputs(rows):
    """GELU keeps its digits where it is small: one input of a row times a weight of one, so
    that the pre-activation h is exact.  h sigmoid(2 u), u = c (h + a h^3): in fp32 the
    roundings of 2 u, a few of 2^-24 of it (with the constants' own 2^-21), are an error of
    25 2^-21 of the exponential where |2 u| is at most 25; the exponential and the division
    add less than 2^-17; in all below 2^-15 of the result, which is rounded once to bf16."""
    h = C.bf16(np.linspace(-6.0, 6.0, rows))
    codes, scales = np.full((1, 8, 32), 8), np.ones((1, 1, 8))
    codes[:, :, 0] = 9
    x = np.zeros((rows, 32))
    x[:, 0] = h
    p = Q4Product(C.device_matrix(codes, scales, 32), act="gelu_tanh")
    got = p.forward(torch.from_numpy(x).bfloat16().cuda(),
                    torch.tensor([0, rows], dtype=torch.int32, device="cuda")).double().cpu().numpy()
    u2 = 2 * np.sqrt(2 / np.pi) * (h + 0.044715 * h ** 3)
    want = (h / (1 + np.exp(-u2)))[:, None]
    assert (np.abs(got - want) <= (C.BF16_HALF + 2.0 ** -14) * np.abs(want)).all(), \
        float((np.abs(got - want) / np.maximum(np.abs(want), 1e-30)).max())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act,bias", [("none", False), ("gelu_tanh", True), ("relu", True), ("swiglu", False)])
def test_product_few_rows_crowded(act, bias, shape):
    """Few rows of many experts, most of them on two: several row tiles of an expert in the
    few-row kernel."""
    N, K, group = shape
    c = _product_case(N + 3 * K, [0, 33, 0, 0, 1, 0, 0, 0, 17, 0], N, K, group, act, bias, before=2, behind=3)
    p, x, off = _device(c)
    out = torch.full((c["R"], N), 7.0, dtype=torch.bfloat16, device="cuda")
    p.forward(x, off, out)
    _check(c, out, fill=7.0)
    assert p.status() == 0


def test_infinite_scale_of_a_short_group_crowded():
    """As test_infinite_scale_of_a_short_group, several row tiles of an expert in the few-row
    kernel."""
    c = _product_case(20, [40, 0, 0, 0, 9, 0, 0, 0], 72, 160, 64, "none", False)
    codes, scales = c["m"][0].copy(), c["m"][1].copy()
    codes[:, 5, 128:] = np.maximum(codes[:, 5, 128:], 9)
    c["x"], c["m"] = C.bf16(np.abs(c["x"]) + 2.0 ** -8), (codes, scales)
    p, x, off = _device(c)
    want = p.forward(x, off)
    _check(c, want)
    scales = scales.copy()
    scales[:, 2, 5] = np.inf
    got = Q4Product(C.device_matrix(codes, scales, 64)).forward(x, off)
    rest = [i for i in range(72) if i != 5]
    assert torch.equal(got[:, rest], want[:, rest]) and bool((got[:, 5] == float("inf")).all())


def test_product_gelu_of_negative_inputs_few_rows():
    """As test_product_gelu_of_negative_inputs, with its bound, in the few-row kernel: the rows
    of one of eight experts."""
    h = C.bf16(np.linspace(-6.0, -2.0, 90))
    codes, scales = np.full((8, 8, 32), 8), np.ones((8, 1, 8))
    codes[:, :, 0] = 9
    x = np.zeros((90, 32))
    x[:, 0] = h
    p = Q4Product(C.device_matrix(codes, scales, 32), act="gelu_tanh")
    off = torch.tensor([0, 0, 0] + [90] * 6, dtype=torch.int32, device="cuda")
    got = p.forward(torch.from_numpy(x).bfloat16().cuda(), off).double().cpu().numpy()
    u2 = 2 * np.sqrt(2 / np.pi) * (h + 0.044715 * h ** 3)
    want = (h / (1 + np.exp(-u2)))[:, None]
    assert (np.abs(got - want) <= (C.BF16_HALF + 2.0 ** -14) * np.abs(want)).all()


def test_product_keeps_little_memory():
    """Calls of many numbers of rows leave no more than 32 MB behind, whatever the outputs."""
    p = Q4Product(quantize(torch.randn(1, 1 << 17, 32, device="cuda"), 32))
    x = torch.randn(64, 32, device="cuda").bfloat16()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for R in range(1, 41):
        out = p.forward(x[:R], torch.tensor([0, R], dtype=torch.int32, device="cuda"))
        assert out.shape == (R, 1 << 17)
    del out
    assert torch.cuda.memory_allocated() - before <= 32 << 20
    assert p.status() == 0

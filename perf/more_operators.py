"""Measurement cases of the operators on 4-bit expert weights: quantising weights
and reading them back, the MoE layer for a few tokens, and the matrix product
grouped by expert over ragged rows.

``own = False`` computes each operator in its plain form, with elementary torch
operations; ``own = True`` makes the calls a program makes of this package.
The expert shapes are those of ``workloads.py``.

A 4-bit matrix [E, N, K] (N outputs, K inputs of each of E experts) is held as
  codes  uint8 [E, N, K / 2]: eight inputs to a 32-bit word, input i of the eight in
         the four bits from 4 (i / 2) + 16 (i % 2) on;
  scales bf16 [E, ceil(K / group), N]: one for `group` inputs of an output;
and stands for w = (code - 8) scale.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def _quant(name, E, N, K, group, dtype):
    case = dict(op="quantize", E=E, N=N, K=K, group=group, dtype=dtype)
    return dict(case, name=name) if name else case


def _decode(name, T, D, F, E, k, act, group, score="softmax", groups=1, top_groups=1, bias=False,
            zipf=0.0, corr=0.0, shared=0, capacity=0.0):
    case = dict(op="decode", T=T, D=D, F=F, E=E, k=k, act=act, group=group, score=score,
                groups=groups, top_groups=top_groups, bias=bias, zipf=zipf, corr=corr,
                shared=shared, capacity=capacity)
    return dict(case, name=name) if name else case


def _product(name, R, E, N, K, group, act, bias=False, zipf=0.0):
    case = dict(op="product", R=R, E=E, N=N, K=K, group=group, act=act, bias=bias, zipf=zipf)
    return dict(case, name=name) if name else case


def listed():
    return [
        # the fp32 weights of a small layer, a group of 32
        _quant("quantize dense fp32", 8, 1024, 512, 32, "f32"),
        # one matrix of every expert of the large layer
        _quant("quantize large", 128, 2048, 4096, 128, "bf16"),
        # one sequence being generated: a small layer with group-limited routing ...
        _decode("decode grouped T1", 1, 1024, 704, 64, 6, "swiglu", 64, "sigmoid", 8, 4, corr=0.1),
        # ... and the large layer, bound by reading eight experts
        _decode("decode large T1", 1, 4096, 2048, 128, 8, "swiglu", 128),
        # a few sequences on a layer with biases
        _decode("decode dense T5", 5, 512, 1024, 8, 2, "gelu_tanh", 32, bias=True),
        # tokens that crowd on few experts, and a shared branch
        _decode("decode skewed T24", 24, 2048, 1408, 64, 8, "swiglu", 128, zipf=1.2, shared=1),
        # the most tokens a call takes: nearly every expert of the large layer is read
        _decode("decode large T64", 64, 4096, 2048, 128, 8, "swiglu", 32),
        # one row by one matrix: a matrix-vector product and nothing else
        _product("product one row", 1, 1, 4096, 2048, 64, "none"),
        # four tokens' assignments over the experts of the grouped layer
        _product("product grouped up R24", 24, 64, 704, 1024, 64, "swiglu"),
        # an odd number of rows of a layer with biases, a last group that is short
        _product("product biased odd", 333, 8, 1000, 480, 64, "gelu_tanh", bias=True),
        # a prompt whose rows crowd on few experts
        _product("product skewed up", 8192, 64, 1408, 2048, 128, "swiglu", zipf=1.2),
        # a batch of prompts on the large layer
        _product("product large up", 32768, 128, 2048, 4096, 64, "swiglu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "decode", "decode", "product", "product", "product"])
    group = rng.choice([32, 64, 128])
    if op == "quantize":
        N, K = 8 * _log(rng, 1, 512), 32 * _log(rng, 1, 256)
        E = max(1, min(_log(rng, 1, 128), (1 << 30) // (N * K)))
        return _quant(None, E, N, K, group, rng.choice(["bf16", "f32"]) if E * N * K < 1 << 29 else "bf16")
    if op == "decode":
        act = rng.choice(["swiglu", "swiglu", "gelu_tanh", "relu"])
        E = rng.choice([8, 16, 24, 64, 96, 128])
        groups = rng.choice([1, 1, 1, 2, 4])
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, top * (E // groups)))
        T = _log(rng, 1, 64)
        D, F = 32 * _log(rng, 1, 128), 32 * _log(rng, 2, 64)
        zipf = rng.choice([0.0, 0.0, 1.2]) if k <= 4 and groups == 1 else 0.0
        return _decode(None, T, D, F, E, k, act, group, rng.choice(["softmax", "sigmoid"]), groups,
                       top, bias=act != "swiglu" and rng.random() < 0.7, zipf=zipf,
                       corr=rng.choice([0.0, 0.1]) if zipf == 0 else 0.0,
                       shared=rng.choice([0, 0, 1, 2]) if act == "swiglu" else 0,
                       capacity=rng.choice([0.0, 0.0, 0.0, 1.25]))
    act = rng.choice(["swiglu", "none", "none", "gelu_tanh", "relu"])
    E = rng.choice([1, 5, 8, 24, 64, 128])
    N, K = 8 * _log(rng, 4, 512), 32 * _log(rng, 1, 128)
    R = _log(rng, 1, 32768)
    mats = 2 if act == "swiglu" else 1
    R = max(1, min(R, (1 << 38) // (N * K * mats)))
    return _product(None, R, E, N, K, group, act, bias=act != "swiglu" and rng.random() < 0.6,
                    zipf=rng.choice([0.0, 1.2]) if E > 1 else 0.0)


# ---- inputs

def _group_amax(w, group):
    """Largest magnitude of each group of inputs: [..., N, ceil(K / group)]."""
    K = w.shape[-1]
    pad = -K % group
    a = w.abs()
    if pad:
        a = torch.nn.functional.pad(a, (0, pad))
    return a.unflatten(-1, (-1, group)).amax(-1)


def _round_up_5_bits(s):
    """The smallest value of five significant bits that is not below s >= 0 (fp32)."""
    bits = (s.view(torch.int32) + 0x7FFFF) & ~0x7FFFF
    return bits.view(torch.float32)


def _quantize(w, group):
    """(q [.., N, K] in -7 .. 7 in w's type, scale [.., N, groups] fp32).  A quotient of
    fp32 weights may fall next to the border of two codes: 64 bits decide there; those
    of bf16 weights (8 bits by 5) are apart from it in 32 bits."""
    amax = _group_amax(w, group).float()
    scale = _round_up_5_bits(amax / torch.full_like(amax, 7.0))    # (a number would multiply by 1 / 7)
    wide = torch.float64 if w.dtype == torch.float32 else torch.float32
    s = scale.to(wide).repeat_interleave(group, -1)[..., :w.shape[-1]]
    q = torch.where(s > 0, torch.round(w.to(wide) / s), 0.0)
    return q, scale


def _pack(q):
    """Codes of q in -8 .. 7 [.., K] as uint8 [.., K / 2]."""
    c = (q + 8).to(torch.uint8).unflatten(-1, (-1, 8))
    low, high = c[..., [0, 4, 1, 5]], c[..., [2, 6, 3, 7]]
    return (low | (high << 4)).flatten(-2)


def _matrix(normal, E, N, K, group, std):
    """A quantised matrix of normally distributed weights, in blocks of experts."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, -(-K // group), N, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // (N * K))
    for e in range(0, E, step):
        w = normal((min(step, E - e), N, K), std, torch.bfloat16)
        q, s = _quantize(w, group)
        codes[e:e + step] = _pack(q)
        scales[e:e + step] = s.transpose(-1, -2).to(torch.bfloat16)
    return codes, scales, group


def _experts_empty(c):
    """Experts that a skewed layer's logit bias never routes to."""
    return min(4, c["E"] - c["k"]) if c["zipf"] > 0 else 0


def _row_shares(c):
    """Probabilities of an expert of rank 0, 1, .. to get a row."""
    w = [(r + 1) ** -c["zipf"] for r in range(c["E"])]
    return [v / sum(w) for v in w]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    c = dict(case)
    s = dict(case=c)
    if c["op"] == "quantize":
        # trained weights: some outputs are wider than the rest
        w = normal((c["E"], c["N"], c["K"]), c["K"] ** -0.5, _DT[c["dtype"]])
        w.mul_(1.0 + 2.0 * (torch.rand(c["E"], c["N"], 1, generator=g, device="cuda") < 0.05))
        s["w"] = w
        return s
    if c["op"] == "product":
        R, E, N, K, group = c["R"], c["E"], c["N"], c["K"], c["group"]
        s["w"] = _matrix(normal, E, N, K, group, K ** -0.5)
        s["w3"] = _matrix(normal, E, N, K, group, K ** -0.5) if c["act"] == "swiglu" else None
        s["bias"] = normal((E, N), 0.1) if c["bias"] else None
        s["x"] = normal((R, K)).bfloat16()
        rng = np.random.default_rng(seed)
        counts = np.zeros(E, np.int64)
        counts[rng.permutation(E)] = rng.multinomial(R, _row_shares(c))
        s["counts"] = counts.tolist()
        s["offsets"] = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device="cuda")
        if own:
            from sparse_mixture_experts_softmax_gb300.q4 import Q4Matrix, Q4Product
            s["product"] = Q4Product(Q4Matrix(*s["w"]), None if s["w3"] is None else Q4Matrix(*s["w3"]),
                                     bias=s["bias"], act=c["act"])
        return s
    T, D, F, E, group = c["T"], c["D"], c["F"], c["E"], c["group"]
    swiglu = c["act"] == "swiglu"
    # normalised tokens, as they come out of the norm in front of the layer
    s["x"] = normal((T, D)).bfloat16()
    s["w_gate"] = normal((E, D), D ** -0.5)
    s["w1"] = _matrix(normal, E, F, D, group, D ** -0.5)
    s["w3"] = _matrix(normal, E, F, D, group, D ** -0.5) if swiglu else None
    s["w2"] = _matrix(normal, E, D, F, group, F ** -0.5)
    s["b1"] = normal((E, F), 0.1) if c["bias"] else None
    s["b2"] = normal((E, D), 0.1) if c["bias"] else None
    s["logit_bias"] = s["corr_bias"] = s["ws1"] = s["ws3"] = s["ws2"] = None
    if c["zipf"] > 0:
        rank = torch.randperm(E, generator=g, device="cuda")
        lb = -c["zipf"] * torch.log(rank.float() + 1)
        s["logit_bias"] = torch.where(rank < E - _experts_empty(c), lb, -math.inf)
    if c["corr"] > 0:
        s["corr_bias"] = (torch.rand(E, generator=g, device="cuda") * 2 - 1) * c["corr"]
    if c["shared"]:
        Fs = c["shared"] * F
        s["ws1"] = _matrix(normal, 1, Fs, D, group, D ** -0.5)
        s["ws3"] = _matrix(normal, 1, Fs, D, group, D ** -0.5)
        s["ws2"] = _matrix(normal, 1, D, Fs, group, Fs ** -0.5)
    if own:
        from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder
        from sparse_mixture_experts_softmax_gb300.q4 import Q4Matrix
        q = {name: None if s[name] is None else Q4Matrix(*s[name])
             for name in ("w1", "w3", "w2", "ws1", "ws3", "ws2")}
        s["decoder"] = MoEDecoder(
            s["w_gate"], q["w1"], q["w2"], w3=q["w3"], b1=s["b1"], b2=s["b2"], k=c["k"],
            act=c["act"], score=c["score"], n_groups=c["groups"], topk_groups=c["top_groups"],
            logit_bias=s["logit_bias"], corr_bias=s["corr_bias"], n_shared=c["shared"],
            ws1=q["ws1"], ws3=q["ws3"], ws2=q["ws2"], capacity_factor=c["capacity"], max_tokens=T)
    return s


# ---- one pass

def run(s):
    op = s["case"]["op"]
    if op == "decode":
        if own:
            d = s["decoder"]
            y = d.decode(s["x"])
            return dict(y=y, idx=d.idx, gate=d.gate)
        return _plain_decode(s)
    if op == "product":
        if own:
            return dict(c=s["product"].forward(s["x"], s["offsets"]))
        return _plain_product(s)
    if own:
        from sparse_mixture_experts_softmax_gb300.q4 import quantize
        q = quantize(s["w"], s["case"]["group"])
        return dict(scales=q.scales, values=q.dequantize())
    return _plain_quantize(s)


def _plain_quantize(s):
    """The values that the codes stand for (exact in bf16: 3 bits by 5) and the scales."""
    c = s["case"]
    q, scale = _quantize(s["w"], c["group"])
    values = q.float() * scale.repeat_interleave(c["group"], -1)[..., :c["K"]]
    return dict(scales=scale.transpose(-1, -2).to(torch.bfloat16).contiguous(),
                values=values.to(torch.bfloat16))


def _plain_weights(matrix, e=slice(None)):
    """Weights [.., N, K] of experts e in 32 bits."""
    codes, scales, group = matrix
    b = codes[e].unflatten(-1, (-1, 4))
    lo, hi = b & 15, b >> 4
    # inputs 0 .. 7 of a word
    c = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2],
                     lo[..., 1], lo[..., 3], hi[..., 1], hi[..., 3]], -1).flatten(-2)
    scale = scales[e].float().transpose(-1, -2).repeat_interleave(group, -1)[..., :c.shape[-1]]
    return (c.float() - 8.0) * scale


def _act(h1, h3, act):
    if act == "swiglu":
        return h1 * torch.sigmoid(h1) * h3
    if act == "none":
        return h1
    if act == "relu":
        return torch.clamp(h1, min=0.0)
    return 0.5 * h1 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (h1 + 0.044715 * h1 ** 3)))


def _plain_product(s):
    c = s["case"]
    out = torch.empty(c["R"], c["N"], dtype=torch.bfloat16, device="cuda")
    r = 0
    for e, n in enumerate(s["counts"]):
        if n == 0:
            continue
        x = s["x"][r:r + n].float()
        h1 = x @ _plain_weights(s["w"], e).t()
        if s["bias"] is not None:
            h1 = h1 + s["bias"][e]
        h3 = x @ _plain_weights(s["w3"], e).t() if s["w3"] is not None else None
        out[r:r + n] = _act(h1, h3, c["act"]).to(torch.bfloat16)
        r += n
    return dict(c=out)


def _plain_route(s):
    """Router in 64 bits: near-equal scores decide whole numbers."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    wg = s["w_gate"].to(s["x"].dtype)      # the layer multiplies with W_g in its own type
    logits = s["x"].double() @ wg.double().t()
    if s["logit_bias"] is not None:
        logits = logits + s["logit_bias"].double()
    if c["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    key = p if s["corr_bias"] is None else p + s["corr_bias"].double()
    if G > 1:
        per = key.view(T, G, E // G).sort(dim=2, descending=True).values
        group = per[:, :, :2].sum(2)
        rank = group.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        keep = (rank < c["top_groups"]).repeat_interleave(E // G, 1)
        key = torch.where(keep, key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    sel = p.gather(1, idx)
    return idx, (sel / sel.sum(1, keepdim=True)).float()


def _plain_decode(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["x"].float()
    idx, gate = _plain_route(s)
    used = gate
    if c["capacity"] > 0:
        # an expert keeps its first assignments in token order
        hot = (idx.reshape(-1, 1) == torch.arange(E, device=x.device)).long()
        place = (hot.cumsum(0) - hot).gather(1, idx.reshape(-1, 1)).view(T, k)
        cap = math.ceil(float(np.float32(c["capacity"])) * T * k / E)
        used = torch.where(place < cap, gate, 0.0)
    if T * k <= E:      # each assignment reads its own expert
        e = idx.reshape(-1)
        xs = x.repeat_interleave(k, 0)[:, :, None]
        h1 = (_plain_weights(s["w1"], e) @ xs)[:, :, 0]
        if s["b1"] is not None:
            h1 = h1 + s["b1"][e]
        h3 = (_plain_weights(s["w3"], e) @ xs)[:, :, 0] if s["w3"] is not None else None
        ye = (_plain_weights(s["w2"], e) @ _act(h1, h3, c["act"])[:, :, None])[:, :, 0]
        if s["b2"] is not None:
            ye = ye + s["b2"][e]
        y = (ye.view(T, k, -1) * used[:, :, None]).sum(1)
    else:               # every expert for every token, weighted by the gates
        h1 = x @ _plain_weights(s["w1"]).transpose(1, 2)
        if s["b1"] is not None:
            h1 = h1 + s["b1"][:, None, :]
        h3 = x @ _plain_weights(s["w3"]).transpose(1, 2) if s["w3"] is not None else None
        ye = _act(h1, h3, c["act"]) @ _plain_weights(s["w2"]).transpose(1, 2)
        if s["b2"] is not None:
            ye = ye + s["b2"][:, None, :]
        w = torch.zeros(T, E, device=x.device).scatter_(1, idx, used)
        y = (ye * w.t()[:, :, None]).sum(0)
    if c["shared"]:
        hs = _act(x @ _plain_weights(s["ws1"], 0).t(), x @ _plain_weights(s["ws3"], 0).t(), "swiglu")
        y = y + hs @ _plain_weights(s["ws2"], 0).t()
    return dict(y=y.to(s["x"].dtype), idx=idx.to(torch.int32), gate=gate)


# ---- the definition in 64 bits

# first bit of each of a word's eight inputs
_PLACE = [4 * (i // 2) + 16 * (i % 2) for i in range(8)]


def _exact_weights(matrix, e):
    """Weights [N, K] of expert e in 64 bits."""
    codes, scales, group = matrix
    words = codes[e].contiguous().view(torch.int32).to(torch.int64)
    K = words.shape[1] * 8
    w = torch.empty(words.shape[0], K, dtype=torch.float64, device=words.device)
    for i, at in enumerate(_PLACE):
        w[:, i::8] = ((words >> at) % 16 - 8).double()
    of = torch.arange(K, device=words.device) // group
    return w.mul_(scales[e].double().t()[:, of])


def _exact_act(a, b, act):
    if act == "swiglu":
        return a / (1 + torch.exp(-a)) * b
    if act == "relu":
        return torch.where(a > 0, a, 0.0)
    if act == "none":
        return a
    return a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "decode":
        return _exact_decode(c, s)
    if c["op"] == "product":
        out = torch.empty(c["R"], c["N"], dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(c["E"]):
            x = s["x"][off[e]:off[e + 1]].double()
            if len(x) == 0:
                continue
            a = torch.einsum("rk,nk->rn", x, _exact_weights(s["w"], e))
            if s["bias"] is not None:
                a += s["bias"][e].double()
            b = torch.einsum("rk,nk->rn", x, _exact_weights(s["w3"], e)) if s["w3"] else None
            out[off[e]:off[e + 1]] = _exact_act(a, b, c["act"])
        return dict(c=out)
    G, K = c["group"], c["K"]
    scales = torch.empty(c["E"], -(-K // G), c["N"], dtype=torch.float64, device="cuda")
    values = torch.empty(c["E"], c["N"], K, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        w = s["w"][e].double()
        for j in range(scales.shape[1]):
            part = w[:, j * G:(j + 1) * G]
            least = part.abs().max(1).values / 7
            m, x = torch.frexp(least)               # m in [1/2, 1): five bits are m 32
            sc = torch.ceil(m * 32) * (x.long() - 5 + 1023 << 52).view(torch.float64)
            scales[e, j] = sc
            values[e, :, j * G:(j + 1) * G] = torch.where(
                sc[:, None] > 0, torch.round(part / sc[:, None]) * sc[:, None], 0.0)
    return dict(scales=scales, values=values)


def _exact_decode(c, s):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = s["x"].double()
    wg = s["w_gate"].to(s["x"].dtype).double()
    logits = torch.stack([wg @ x[t] for t in range(T)]).cpu().numpy()
    if s["logit_bias"] is not None:
        logits = logits + s["logit_bias"].double().cpu().numpy()
    cb = s["corr_bias"].double().cpu().numpy() if s["corr_bias"] is not None else np.zeros(E)
    cap = math.inf
    if c["capacity"] > 0:
        cap = math.ceil(float(np.float32(c["capacity"])) * T * k / E)
    rows = [[] for _ in range(E)]           # (token, gate) of the assignments an expert keeps
    idx, gate = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        if c["score"] == "softmax":
            p = np.exp(logits[t] - logits[t].max())
            p /= p.sum()
        else:
            p = 1 / (1 + np.exp(-logits[t]))
        key = p + cb
        allowed = range(E)
        if G > 1:
            n = E // G
            best = [sum(sorted(key[q * n:(q + 1) * n])[-2:]) for q in range(G)]
            kept = sorted(range(G), key=lambda q: (-best[q], q))[:c["top_groups"]]
            allowed = [e for e in range(E) if e // n in kept]
        chosen = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        total = sum(p[e] for e in chosen)
        for j, e in enumerate(chosen):
            idx[t, j], gate[t, j] = e, p[e] / total
            if len(rows[e]) < cap:
                rows[e].append((t, p[e] / total))
    y = torch.zeros(T, c["D"], dtype=torch.float64, device="cuda")

    def branch(w1, w3, w2, e, xs):
        a = xs @ _exact_weights(w1, e).t()
        if s["b1"] is not None:
            a = a + s["b1"][e].double()
        a = _exact_act(a, xs @ _exact_weights(w3, e).t() if w3 else None, c["act"])
        v = a @ _exact_weights(w2, e).t()
        return v if s["b2"] is None else v + s["b2"][e].double()

    for e in range(E):
        if rows[e]:
            t = torch.tensor([r[0] for r in rows[e]], device="cuda")
            w = torch.tensor([r[1] for r in rows[e]], dtype=torch.float64, device="cuda")
            y.index_add_(0, t, w[:, None] * branch(s["w1"], s["w3"], s["w2"], e, x[t]))
    if c["shared"]:
        y += branch(s["ws1"], s["ws3"], s["ws2"], 0, x)
    return dict(y=y, idx=idx, gate=gate)


# ---- what a pass cannot do without

def _matrix_bytes(N, K, group):
    return N * K / 2 + 2 * N * -(-K // group)


def _experts_read(c):
    """Expected number of distinct experts that T tokens choose."""
    E, k, T = c["E"], c["k"], c["T"]
    if c["zipf"] > 0:
        w = [(r + 1) ** -c["zipf"] for r in range(E - _experts_empty(c))]
        p = [min(1.0, k * v / sum(w)) for v in w]
    else:
        p = [k / E] * E
    return max(min(k, E), sum(1 - (1 - q) ** T for q in p))


def work(case):
    c = case
    if c["op"] == "quantize":
        n, q = c["E"] * c["N"] * c["K"], c["E"] * _matrix_bytes(c["N"], c["K"], c["group"])
        # weights in, codes and scales out; codes and scales in, bf16 values out
        return dict(bytes=n * (_SIZE[c["dtype"]] + 2) + 2 * q, flops=6 * n)
    if c["op"] == "product":
        R, N, K, mats = c["R"], c["N"], c["K"], 2 if c["act"] == "swiglu" else 1
        read = sum(1 - (1 - p) ** R for p in _row_shares(c))
        nbytes = read * (mats * _matrix_bytes(N, K, c["group"]) + (4 * N if c["bias"] else 0))
        return dict(bytes=nbytes + 2 * R * (N + K) + 4 * (c["E"] + 1), flops=2 * R * N * K * mats)
    T, D, F, E, k = c["T"], c["D"], c["F"], c["E"], c["k"]
    up = 2 if c["act"] == "swiglu" else 1
    expert = up * _matrix_bytes(F, D, c["group"]) + _matrix_bytes(D, F, c["group"])
    nbytes = _experts_read(c) * (expert + (4 * (F + D) if c["bias"] else 0))
    nbytes += 4 * E * D + c["shared"] * expert + 4 * T * D + 8 * T * k
    flops = 2 * T * (E * D + (k * (up + 1) + 3 * c["shared"]) * F * D)
    return dict(bytes=nbytes, flops=flops)

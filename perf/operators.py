"""Measurement cases of the pre-norm MoE block's operators: the layer norm with
its residual add (forward and backward) and the MoE layer for a few tokens.

``own = False`` computes each operator in its plain form, with elementary torch
operations; ``own = True`` makes the calls a program makes of this package.
The expert shapes are those of ``workloads.py``.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def _decode(name, T, D, F, E, k, act, dtype, score="softmax", groups=1, top_groups=1, bias=False,
            zipf=0.0, corr=0.0, shared=0, capacity=0.0):
    case = dict(op="decode", T=T, D=D, F=F, E=E, k=k, act=act, dtype=dtype, score=score,
                groups=groups, top_groups=top_groups, bias=bias, zipf=zipf, corr=corr,
                shared=shared, capacity=capacity)
    return dict(case, name=name) if name else case


def _norm(name, op, T, D, x, z="bf16", delta="none", stats=True, bias=True, res=True):
    if op == "norm":
        case = dict(op=op, T=T, D=D, x=x, delta=delta, z=z, stats=stats, bias=bias)
    else:
        case = dict(op=op, T=T, D=D, x=x, bias=bias, res=res)
    return dict(case, name=name) if name else case


def listed():
    return [
        # the smallest layer there is, one token: launch latency and nothing else
        _decode("decode tiny fp32 T1", 1, 32, 64, 4, 2, "relu", "f32", bias=True),
        # one sequence being generated: a small layer with group-limited routing ...
        _decode("decode grouped T1", 1, 1024, 704, 64, 6, "swiglu", "bf16", "sigmoid", 8, 4,
                corr=0.1),
        # ... and the large layer, bound by reading eight experts
        _decode("decode large T1", 1, 4096, 2048, 128, 8, "swiglu", "bf16"),
        # a few sequences, with shared experts; a batch whose tokens crowd on few experts
        _decode("decode shared T7", 7, 1024, 704, 64, 6, "swiglu", "bf16", "sigmoid", 8, 4,
                shared=2),
        _decode("decode skewed T24", 24, 2048, 1408, 64, 8, "swiglu", "bf16", zipf=1.2),
        # an fp32 layer with biases
        _decode("decode dense fp32 T13", 13, 512, 1024, 8, 2, "gelu_tanh", "f32", bias=True),
        # the most tokens a call takes: nearly every expert of the large layer is read
        _decode("decode large T64", 64, 4096, 2048, 128, 8, "swiglu", "bf16"),
        # the residual add and norm of one token between two layers
        _norm("norm T1", "norm", 1, 4096, "bf16", "bf16", "bf16", stats=False),
        # a training batch of the large layer: bf16 stream, the layer's fp32 output added
        _norm("norm train", "norm", 65536, 4096, "bf16", "bf16", "f32"),
        # an odd width and an odd number of rows, fp32 stream into a bf16 layer, no add
        _norm("norm odd", "norm", 5003, 1023, "f32", "bf16"),
        # gradients of a small fp32 layer's batch, and of the large layer's
        _norm("norm backward small", "norm_bwd", 4096, 512, "f32"),
        _norm("norm backward train", "norm_bwd", 65536, 4096, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "norm", "norm_bwd"])
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        act = rng.choice(["swiglu", "swiglu", "gelu_tanh", "relu"])
        E = rng.choice([8, 16, 24, 64, 96, 128] + ([4, 6, 20] if dtype == "f32" else []))
        groups = rng.choice([1, 1, 1, 2, 4]) if E >= 8 and E % 4 == 0 else 1
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, top * (E // groups)))
        T = _log(rng, 1, 64)
        D, F = 8 * _log(rng, 4, 512), 8 * _log(rng, 8, 256)
        while E * D * F * (3 if act == "swiglu" else 2) * _SIZE[dtype] > 6.4e9:
            F = max(64, F // 16 * 8)
        zipf = rng.choice([0.0, 0.0, 1.2]) if k <= 4 and groups == 1 else 0.0
        return _decode(None, T, D, F, E, k, act, dtype, rng.choice(["softmax", "sigmoid"]), groups,
                       top, bias=act != "swiglu" and rng.random() < 0.7,
                       zipf=zipf, corr=rng.choice([0.0, 0.1]) if zipf == 0 else 0.0,
                       shared=rng.choice([0, 0, 1, 2]) if act == "swiglu" and dtype == "bf16" else 0,
                       capacity=rng.choice([0.0, 0.0, 0.0, 1.25]))
    D = _log(rng, 16, 8192) if rng.random() < 0.5 else 8 * _log(rng, 2, 1024)
    T = min(_log(rng, 1, 65536), (1 << 28) // D)
    x = rng.choice(["bf16", "f32"])
    if op == "norm":
        return _norm(None, op, T, D, x, rng.choice(["bf16", "f32"]),
                     rng.choice(["none", "bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.7)
    return _norm(None, op, T, D, x, bias=rng.random() < 0.7, res=rng.random() < 0.7)


# ---- inputs

def _experts_empty(c):
    """Experts that a skewed layer's logit bias never routes to."""
    return min(4, c["E"] - c["k"]) if c["zipf"] > 0 else 0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    c = dict(case)
    T, D = c["T"], c["D"]
    s = dict(case=c)
    if c["op"] == "decode":
        F, E, dt = c["F"], c["E"], _DT[c["dtype"]]
        swiglu = c["act"] == "swiglu"
        # normalised tokens, as they come out of the norm in front of the layer
        s["x"] = normal((T, D)).to(dt)
        s["w_gate"] = normal((E, D), D ** -0.5)
        s["w1"] = normal((E, F, D), D ** -0.5, dt)
        s["w3"] = normal((E, F, D), D ** -0.5, dt) if swiglu else None
        s["w2"] = normal((E, D, F), F ** -0.5, dt)
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
            s["ws1"], s["ws3"] = normal((Fs, D), D ** -0.5, dt), normal((Fs, D), D ** -0.5, dt)
            s["ws2"] = normal((D, Fs), Fs ** -0.5, dt)
        if own:
            from sparse_mixture_experts_softmax_gb300.decode import MoEDecoder
            s["decoder"] = MoEDecoder(
                s["w_gate"], s["w1"], s["w2"], w3=s["w3"], b1=s["b1"], b2=s["b2"], k=c["k"],
                act=c["act"], score=c["score"], n_groups=c["groups"], topk_groups=c["top_groups"],
                logit_bias=s["logit_bias"], corr_bias=s["corr_bias"], n_shared=c["shared"],
                ws1=s["ws1"], ws3=s["ws3"], ws2=s["ws2"], capacity_factor=c["capacity"],
                max_tokens=T)
        return s
    # a residual stream: a common offset, and channels that are wider than the rest
    scale = 1.0 + 4.0 * (torch.rand(D, generator=g, device="cuda") < 0.02).float()
    h = normal((T, D))
    h.mul_(scale).add_(0.25)
    s["x"] = h.to(_DT[c["x"]])
    s["gamma"] = 1.0 + normal((D,), 0.1)
    s["beta"] = normal((D,), 0.1) if c["bias"] else None
    s["delta"] = None
    if c["op"] == "norm":
        if c["delta"] != "none":
            s["delta"] = normal((T, D), 0.5).to(_DT[c["delta"]])
    else:
        s["dz"] = normal((T, D), 1.0 / math.sqrt(T))
        s["dres"] = normal((T, D), 1.0 / math.sqrt(T)) if c["res"] else None
        # what the forward pass has left
        s["mean"] = torch.empty(T, device="cuda")
        s["rstd"] = torch.empty(T, device="cuda")
        for r in range(0, T, 8192):
            v = s["x"][r:r + 8192].double()
            s["mean"][r:r + 8192] = v.mean(1)
            s["rstd"][r:r + 8192] = (v.var(1, unbiased=False) + _EPS).rsqrt()
    if own:
        from sparse_mixture_experts_softmax_gb300.norm import LayerNorm
        s["norm"] = LayerNorm(s["gamma"], s["beta"], x_dtype=c["x"], z_dtype=c.get("z", "bf16"),
                              eps=_EPS)
    return s


_EPS = 1e-5


# ---- one pass

def run(s):
    op = s["case"]["op"]
    if op == "decode":
        if own:
            d = s["decoder"]
            y = d.decode(s["x"])
            return dict(y=y, idx=d.idx, gate=d.gate)
        return _plain_decode(s)
    if op == "norm":
        if own:
            r = s["norm"].forward(s["x"], s["delta"], stats=s["case"]["stats"])
            return dict(h=r.h, z=r.z, mean=r.mean, rstd=r.rstd)
        return _plain_norm(s)
    if own:
        r = s["norm"].backward(s["dz"], s["x"], s["mean"], s["rstd"], dres=s["dres"])
        return dict(dx=r.dx, dgamma=r.dgamma, dbeta=r.dbeta)
    return _plain_norm_bwd(s)


def _plain_norm(s):
    c = s["case"]
    h = s["x"]
    if s["delta"] is not None:
        h = (h.float() + s["delta"].float()).to(h.dtype)
    v = h.float()
    mean = v.mean(1)
    d = v - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + _EPS)
    z = d * rstd[:, None] * s["gamma"]
    if s["beta"] is not None:
        z = z + s["beta"]
    return dict(h=h if s["delta"] is not None else None, z=z.to(_DT[c["z"]]),
                mean=mean if c["stats"] else None, rstd=rstd if c["stats"] else None)


def _plain_norm_bwd(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = s["dz"] * s["gamma"]
    dx = g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"]
    return dict(dx=dx, dgamma=(s["dz"] * xh).sum(0),
                dbeta=s["dz"].sum(0) if s["beta"] is not None else None)


def _act(h1, h3, act):
    if act == "swiglu":
        return h1 * torch.sigmoid(h1) * h3
    if act == "relu":
        return torch.clamp(h1, min=0.0)
    return 0.5 * h1 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (h1 + 0.044715 * h1 ** 3)))


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
        h1 = (s["w1"][e].float() @ xs)[:, :, 0]
        if s["b1"] is not None:
            h1 = h1 + s["b1"][e]
        h3 = (s["w3"][e].float() @ xs)[:, :, 0] if s["w3"] is not None else None
        ye = (s["w2"][e].float() @ _act(h1, h3, c["act"])[:, :, None])[:, :, 0]
        if s["b2"] is not None:
            ye = ye + s["b2"][e]
        y = (ye.view(T, k, -1) * used[:, :, None]).sum(1)
    else:               # every expert for every token, weighted by the gates
        h1 = x @ s["w1"].float().transpose(1, 2)
        if s["b1"] is not None:
            h1 = h1 + s["b1"][:, None, :]
        h3 = x @ s["w3"].float().transpose(1, 2) if s["w3"] is not None else None
        ye = _act(h1, h3, c["act"]) @ s["w2"].float().transpose(1, 2)
        if s["b2"] is not None:
            ye = ye + s["b2"][:, None, :]
        w = torch.zeros(T, E, device=x.device).scatter_(1, idx, used)
        y = (ye * w.t()[:, :, None]).sum(0)
    if c["shared"]:
        hs = _act(x @ s["ws1"].float().t(), x @ s["ws3"].float().t(), "swiglu")
        y = y + hs @ s["ws2"].float().t()
    return dict(y=y.to(s["x"].dtype), idx=idx.to(torch.int32), gate=gate)


# ---- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "decode":
        return _exact_decode(c, s)
    rows = []
    for r in range(0, c["T"], 4096):        # row blocks, to bound the memory
        part = {key: s[key][r:r + 4096] if s.get(key) is not None else None
                for key in ("x", "delta", "dz", "dres", "mean", "rstd")}
        rows.append(_exact_rows(c, s, part))
    out = {}
    for key in rows[0]:
        v = [r[key] for r in rows]
        if v[0] is None:
            out[key] = None
        else:
            out[key] = torch.stack(v).sum(0) if key in ("dgamma", "dbeta") else torch.cat(v)
    return out


def _exact_rows(c, s, p):
    gamma = s["gamma"].double()
    if c["op"] == "norm":
        h = p["x"]
        if p["delta"] is not None:          # the stream is kept in its own type
            h = (h.double() + p["delta"].double()).to(h.dtype)
        var, mean = torch.var_mean(h.double(), dim=1, correction=0)
        rstd = (var + _EPS) ** -0.5
        z = torch.addcmul(s["beta"].double() if s["beta"] is not None else gamma * 0,
                          (h.double() - mean.unsqueeze(1)) * rstd.unsqueeze(1), gamma)
        return dict(h=h if p["delta"] is not None else None, z=z,
                    mean=mean if c["stats"] else None, rstd=rstd if c["stats"] else None)
    D = c["D"]
    m, r = p["mean"].double()[:, None], p["rstd"].double()[:, None]
    dz = p["dz"].double()
    xc = p["x"].double() - m
    u = dz * gamma
    proj = torch.einsum("td,td->t", u, xc)[:, None]
    dx = r * u - r * u.sum(1, keepdim=True) / D - r ** 3 * xc * proj / D
    if p["dres"] is not None:
        dx += p["dres"].double()
    return dict(dx=dx, dgamma=torch.einsum("td,td->d", dz, xc * r),
                dbeta=dz.sum(0) if s["beta"] is not None else None)


def _exact_decode(c, s):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    dt = s["x"].dtype
    x = s["x"].double()
    wg = s["w_gate"].to(dt).double()
    logits = torch.stack([wg @ x[t] for t in range(T)]).cpu().numpy()
    if s["logit_bias"] is not None:
        logits = logits + s["logit_bias"].double().cpu().numpy()
    cb = s["corr_bias"].double().cpu().numpy() if s["corr_bias"] is not None else np.zeros(E)
    cap = math.inf
    if c["capacity"] > 0:
        cap = math.ceil(float(np.float32(c["capacity"])) * T * k / E)
    taken = [0] * E
    idx, gate = np.zeros((T, k), np.int32), np.zeros((T, k))
    y = torch.zeros(T, c["D"], dtype=torch.float64, device="cuda")
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
            taken[e] += 1
            if taken[e] > cap:
                continue
            a = s["w1"][e].double() @ x[t]
            if s["b1"] is not None:
                a = a + s["b1"][e].double()
            if c["act"] == "swiglu":
                a = a / (1 + torch.exp(-a)) * (s["w3"][e].double() @ x[t])
            elif c["act"] == "relu":
                a = torch.where(a > 0, a, 0.0)
            else:
                a = a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
            v = s["w2"][e].double() @ a
            if s["b2"] is not None:
                v = v + s["b2"][e].double()
            y[t] += float(gate[t, j]) * v
        if c["shared"]:
            a = s["ws1"].double() @ x[t]
            a = a / (1 + torch.exp(-a)) * (s["ws3"].double() @ x[t])
            y[t] += s["ws2"].double() @ a
    return dict(y=y, idx=idx, gate=gate)


# ---- what a pass cannot do without

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
    T, D = c["T"], c["D"]
    if c["op"] == "decode":
        F, E, k, es = c["F"], c["E"], c["k"], _SIZE[c["dtype"]]
        mats = 3 if c["act"] == "swiglu" else 2
        read = _experts_read(c)
        nbytes = read * (mats * F * D * es + (4 * (F + D) if c["bias"] else 0))
        nbytes += 4 * E * D + 3 * c["shared"] * F * D * es + 2 * T * D * es + 8 * T * k
        flops = 2 * T * (E * D + k * mats * F * D + 3 * c["shared"] * F * D)
        return dict(bytes=nbytes, flops=flops)
    ex = _SIZE[c["x"]]
    if c["op"] == "norm":
        row = ex + _SIZE[c["z"]] + (ex + _SIZE[c["delta"]] if c["delta"] != "none" else 0)
        return dict(bytes=T * D * row + 8 * D + (8 * T if c["stats"] else 0), flops=8 * T * D)
    return dict(bytes=T * D * (ex + 8 + (4 if c["res"] else 0)) + 12 * D + 8 * T,
                flops=14 * T * D)

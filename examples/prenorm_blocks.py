"""Two pre-norm MoE blocks, trained for a few steps and then served.

    python examples/prenorm_blocks.py [steps]

Training: h -> block 1 -> block 2, a mean-squared loss on the stream behind them,
the backward pass through both blocks and SGD on every parameter.  Serving: the
same weights, a few tokens at a time, the whole stack of calls captured into one
CUDA graph.  Needs a GB300.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import workloads as W  # noqa: E402
from sparse_mixture_experts_softmax_gb300.block import MoEBlock  # noqa: E402
from sparse_mixture_experts_softmax_gb300.layer import MoELayer  # noqa: E402
from sparse_mixture_experts_softmax_gb300.norm import LayerNorm  # noqa: E402


def make_block(wl, seed):
    inp = W.make_inputs(wl, seed=seed, device="cuda", with_target=False)
    layer = MoELayer(wl.T, wl.D, wl.F, wl.E, wl.k, wl.act, wl.score, wl.dtype, wl.has_bias,
                     0.0, inp["w_gate"], inp["w1"], inp["w2"], w3=inp["w3"], b1=inp["b1"],
                     b2=inp["b2"], n_groups=wl.n_groups, topk_groups=wl.topk_groups)
    norm = LayerNorm(torch.ones(wl.D, device="cuda"), torch.zeros(wl.D, device="cuda"),
                     x_dtype="bf16", z_dtype=wl.dtype)
    return MoEBlock(norm, layer)


def sgd(block, lr):
    la, n = block.layer, block.norm
    n.gamma.add_(n.dgamma, alpha=-lr)
    n.beta.add_(n.dbeta, alpha=-lr)
    grads = la.grad_dict()
    for name, p in la.param_dict().items():
        if p is None:
            continue
        p.add_(grads["d" + name], alpha=-lr)
        lp = getattr(la, name + "_lp", None)
        if lp is not None:
            lp.copy_(p)


def train(blocks, h, target, steps, lr):
    losses = []
    for _ in range(steps):
        states, y = [], None
        x = h
        for b in blocks:
            s, y = b.forward(x, y)
            states.append(s)
            x = s.h
        diff = x.float() + y - target
        losses.append(float((diff * diff).mean()))
        d = diff.mul_(2.0 / diff.numel())
        for b, s in zip(reversed(blocks), reversed(states)):
            d = b.backward(s, d)
        for b in blocks:
            sgd(b, lr)
    return losses


def serve(blocks, tokens):
    """The stream behind the stack for a few tokens, from a captured graph."""
    x = tokens.clone()

    def step():
        h, y = x, None
        for b in blocks:
            h, y = b.decode(h, y)
        return h.float() + y.float()

    step()                                  # decoders and buffers are made outside the graph
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    return out


def main(steps=10):
    wl = W.WORKLOADS["grouped"].with_tokens(512)
    blocks = [make_block(wl, seed) for seed in (0, 1)]
    g = torch.Generator("cuda").manual_seed(7)
    h = torch.randn(wl.T, wl.D, device="cuda", generator=g).bfloat16()
    target = h.float() + 0.5 * torch.randn(wl.T, wl.D, device="cuda", generator=g)
    losses = train(blocks, h, target, steps, lr=50.0)
    print("loss", " ".join(f"{v:.4f}" for v in losses))

    # what serving makes of the first tokens, beside the training forward
    x, y = h, None
    for b in blocks:
        s, y = b.forward(x, y)
        x = s.h
    want = (x.float() + y)[:6]
    got = serve(blocks, h[:6].contiguous())
    err = float((got - want).abs().max() / want.abs().max())
    print(f"served 6 tokens: {err:.1e} of the largest value from the training forward")
    return losses, err


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 10)

"""4-bit expert weights in plain numpy (float64): the packed layout, quantising and
the grouped product, written from include/moe_q4.h."""

import math

import numpy as np
import torch

BF16_HALF = 2.0 ** -8       # half a step of a bf16 value, relative to it


def bf16(a):
    """float64 -> the nearest bf16 value (through fp32, exact for what the tests hold)."""
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().double().numpy()


def pack(codes):
    """codes [.., K] of 0 .. 15 -> uint8 [.., K / 2]."""
    c = np.asarray(codes, np.uint32).reshape(*codes.shape[:-1], -1, 8)
    word = np.zeros(c.shape[:-1], np.uint32)
    for i in range(8):
        word |= c[..., i] << np.uint32(4 * (i // 2) + 16 * (i % 2))
    return word.astype("<u4").view(np.uint8).reshape(*codes.shape[:-1], -1)


def unpack(packed):
    word = np.ascontiguousarray(packed).view("<u4")
    c = np.stack([(word >> np.uint32(4 * (i // 2) + 16 * (i % 2))) & 15 for i in range(8)], -1)
    return c.reshape(*packed.shape[:-1], -1)


def quantize(w, group):
    """codes [E, N, K], scales [E, ceil(K / group), N] (float64) of w [E, N, K] (float64)."""
    E, N, K = w.shape
    G = -(-K // group)
    codes = np.full((E, N, K), 8, np.int64)
    scales = np.zeros((E, G, N))
    for g in range(G):
        part = w[:, :, g * group:(g + 1) * group]
        with np.errstate(all="ignore"):
            least = np.abs(part).max(-1) / 7
            m, x = np.frexp(least)
            # five bits; below the normal numbers of fp32 the places stay those of 2^-126
            x = np.maximum(x, -125)
            s = np.ldexp(np.ceil(np.ldexp(least, 5 - x)), x - 5)
            s = np.where(np.isfinite(part).all(-1), s, np.nan)
            q = np.rint(part / s[..., None])
        codes[:, :, g * group:(g + 1) * group] = np.where(s[..., None] > 0, q, 0).astype(np.int64) + 8
        scales[:, g] = s
    return codes, scales


def weights(codes, scales, group):
    """(code - 8) scale rounded to bf16, [E, N, K]."""
    K = codes.shape[-1]
    s = np.repeat(scales, group, axis=1)[:, :K].transpose(0, 2, 1)
    with np.errstate(all="ignore"):
        return bf16((codes - 8.0) * s)


def random_matrix(rng, E, N, K, group, five_bits=True):
    """codes over all of 0 .. 15 and scales of about 1 / (4 sqrt(K)); their product has
    weights of a standard deviation of about 1 / sqrt(K)."""
    codes = rng.integers(0, 16, (E, N, K))
    s = np.exp(rng.normal(0, 0.3, (E, -(-K // group), N))) / (4.6 * math.sqrt(K))
    s = bf16(s)
    if five_bits:
        m, x = np.frexp(s)
        s = np.ldexp(np.rint(m * 32), x - 5)
    return codes, s


def device_matrix(codes, scales, group):
    from sparse_mixture_experts_softmax_gb300.q4 import Q4Matrix
    return Q4Matrix(torch.from_numpy(pack(codes)).cuda(),
                    torch.from_numpy(scales).float().bfloat16().cuda().contiguous(), group)


def act_of(name, h1, h3):
    if name == "none":
        return h1
    if name == "relu":
        return np.where(h1 < 0, 0.0, h1)
    if name == "gelu_tanh":
        return 0.5 * h1 * (1 + np.tanh(math.sqrt(2 / math.pi) * (h1 + 0.044715 * h1 ** 3)))
    return h1 / (1 + np.exp(-h1)) * h3


def sum_error(x, w):
    """Bound of the error of fp32 sums  x w^T  of K terms: a chain of K / 16 additions
    (16 products at a time, the fewest that a step of the kernels adds) and the 16 within
    one, each off by at most 2^-23 of the partial sum (a rounding with one guard bit
    fewer than the nearest), and partial sums within six times the square root of
    sum (x w)^2, the standard deviation of a sum of terms of random sign."""
    K = x.shape[1]
    return (K / 16 + 16) * 2.0 ** -23 * 6 * np.sqrt((x * x) @ (w * w).T)


def product_row_block(act, x, w, w3=None, bias=None):
    """(values, bound of their error before the rounding) of one expert's rows."""
    h1, e1 = x @ w.T, sum_error(x, w)
    if bias is not None:
        h1 = h1 + bias
        e1 = e1 + 2.0 ** -23 * (np.abs(h1) + np.abs(bias))
    h3, e3 = (x @ w3.T, sum_error(x, w3)) if w3 is not None else (None, 0.0)
    y = act_of(act, h1, h3)
    # the slopes of SiLU and GELU are at most 1.2; their own evaluation in fp32: 2^-18
    if act == "swiglu":
        err = 1.2 * e1 * (np.abs(h3) + e3) + np.abs(h1) * e3
    else:
        err = 1.2 * e1
    return y, err + 2.0 ** -18 * np.abs(y)

"""The decode-step operators over per-head token records, from their
definitions in 64 bits (torch, on whatever device the inputs are), and the
error bounds their tests use.

A record of `heads` key-value heads is [heads * 128 keys][heads * 128 values],
bf16.  Rounding to bf16 is off by at most 2^-8 of the value.
"""
import math

import torch

D = 128
BF16 = 2.0 ** -8


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    """x [n][heads][128] -> (y, size): the normed and rotated heads, and for
    each element the length of the pair it belongs to (its own magnitude
    where nothing rotates)."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    size = y.abs()
    half = len(inv_freq)
    if half:
        i = torch.arange(half, device=x.device)
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = pos.double()[:, None] * torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        a, b = y[..., first], y[..., second]
        y[..., first], y[..., second] = a * c - b * s, a * s + b * c
        size[..., first] = size[..., second] = torch.sqrt(a * a + b * b)
    return y, size


# The kernel's fp32 chain before the final rounding: the sum of 128 squares is
# at most 20 roundings deep (relative 20 * 2^-24), which the square root
# halves; rsqrtf adds 4 * 2^-24, the two products 2 * 2^-24: 16 * 2^-24 =
# 2^-20.  cos and sin: 2^-23 each from sincospif, pi * 2^-25 from its rounded
# argument and 2^-21 from the frequency's 2^-52 at positions up to 2^31;
# two products and a sum add 2 * 2^-24.  A pair (a, b) of length s contributes
# |a| + |b| <= 1.42 s: in all below s * 2^-18.
NORM_ROPE_FP32 = 2.0 ** -18


def norm_rope_bound(y, size):
    return BF16 * y.abs() + NORM_ROPE_FP32 * size


def split(records, heads):
    """(keys, values), each [heads][n][128] fp64, of records [n][heads * 256] bf16."""
    r = records.double().view(-1, 2, heads, D).permute(1, 2, 0, 3)
    return r[0], r[1]


def attention(q, keys, values, scale):
    """q [heads * group][128], keys and values [heads][n][128] ->
    (out [heads * group][128], p [heads * group][n], bound on out's error,
    relative bound on p's error)."""
    heads, n, _ = keys.shape
    q = q.double()
    hq = q.shape[0]
    if n == 0:
        z = torch.zeros((hq, D), dtype=torch.float64, device=q.device)
        return z, torch.zeros((hq, 0), dtype=torch.float64, device=q.device), z, 0.0
    qg = q.view(heads, hq // heads, D)
    s = torch.einsum("hgd,hnd->hgn", qg, keys) * scale
    p = torch.softmax(s, -1)
    out = torch.einsum("hgn,hnd->hgd", p, values).reshape(hq, D)
    weight = torch.einsum("hgn,hnd->hgd", p, values.abs()).reshape(hq, D)
    # a score: 128 exact products summed in fp32, 128 * 2^-23 of the sum of
    # their magnitudes whatever the order and the rounding of an addition, and
    # 4 * 2^-24 of it for the two scalings and the difference from the
    # maximum; exp2f 2^-22
    size = torch.einsum("hgd,hnd->hgn", qg.abs(), keys.abs()).max().item() * abs(scale)
    score = size * (128 * 2.0 ** -23 + 4 * 2.0 ** -24) * 2 + 2.0 ** -22
    # a probability is a quotient of two such, and the sum below it has up to
    # n additions
    rel = 2 * score + n * 2.0 ** -23
    # the output: each probability rounded once to bf16, up to n additions,
    # the result rounded once
    bound = weight * (BF16 + rel + n * 2.0 ** -23) + BF16 * out.abs() * (1 + BF16)
    return out, p.reshape(hq, n), bound, rel


def keep(weights, n, k, recent):
    """The positions kept of the first n of `weights` (a list of floats)."""
    last = min(recent, n)
    w = [-math.inf if math.isnan(x) else x for x in weights[:n - last]]
    heavy = sorted(range(n - last), key=lambda j: (-w[j], j))[:k - last]
    return sorted(heavy) + list(range(n - last, n))

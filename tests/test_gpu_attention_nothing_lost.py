"""hs_prefix_attention and hs_sparse_attention_weights with values that show
what random ones hide in the rounding: a block of keys that is left out or
taken twice, and a probability that is rounded to fewer bits than it should be."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def prefix_attention(q, prefix, P, cache, rows, idx, R, k, hq, h):
    out = torch.full((R, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    need = hs.hs_prefix_attention_bytes(R, hq, h, P, k)
    work = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    hs.hs_prefix_attention(q, prefix, P, cache, rows, idx, R, k, hq, h, SCALE, out, work, need)
    return out


def marked(n, h, block, g):
    """n records whose values are 1 in the dimension of their block of `block`
    rows, another one for each head, and 0 elsewhere; random keys."""
    rec = torch.randn((n, 2, h, 128), generator=g, device="cuda")
    at = torch.arange(n, device="cuda")[:, None] // block + 37 * torch.arange(h, device="cuda")
    rec[:, 1] = torch.nn.functional.one_hot(at % 128, 128).float()
    return rec.to(torch.bfloat16).view(n, h * 256)


def check(q, records, out, h, block):
    """An output is the weight of the blocks of its dimension, all of it
    positive: the bound is 2^-7 of it and the smaller terms of its derivation;
    one block of `parts` or fewer that share a dimension holds far more."""
    keys, values = ref.split(records, h)
    want, _, bound, _ = ref.attention(q, keys, values, SCALE)
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), (err - bound).max().item()
    n = records.shape[0]
    s = torch.einsum("hgd,hnd->hgn", q.double().view(h, -1, 128), keys) * SCALE
    p = torch.softmax(s, -1).reshape(q.shape[0], n)
    pad = -n % block
    mass = torch.nn.functional.pad(p, (0, pad)).view(q.shape[0], -1, block).sum(-1)
    head = torch.arange(q.shape[0], device="cuda") // (q.shape[0] // h)
    dim = (torch.arange(mass.shape[1], device="cuda") + 37 * head[:, None]) % 128
    full = slice(None) if not pad else slice(0, mass.shape[1] - 1)   # (a last short one may be small)
    assert bool((mass > bound.gather(1, dim))[:, full].all())


@pytest.mark.parametrize("R,hq,h,P,block", [
    (2, 8, 8, 517, 64), (19, 12, 4, 20011, 64), (9, 56, 7, 50000, 64), (18, 49, 7, 60000, 64),
    (1, 112, 7, 47001, 64), (3, 3, 1, 70007, 64), (32, 32, 8, 32768, 64), (64, 64, 8, 30011, 128),
    (48, 8, 1, 50001, 128), (33, 42, 7, 90000, 128), (100, 32, 8, 1000, 128), (700, 16, 1, 900, 128)])
def test_every_block_of_the_prefix_counts_once(R, hq, h, P, block):
    g = torch.Generator(device="cuda").manual_seed(P)
    q = torch.randn((R, hq, 128), generator=g, device="cuda").mul(0.5).to(torch.bfloat16)
    prefix = marked(P, h, block, g)
    out = prefix_attention(q, prefix, P, None, 0, None, R, 0, hq, h)
    for r in sorted({0, R // 3, R // 2, R - 1}):
        check(q[r], prefix, out[r], h, block)


@pytest.mark.parametrize("h", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("R,k,group", [(30, 1001, 3), (2, 30000, 9), (160, 40, 1)])
def test_every_tile_of_published_rows_counts_once(R, k, group, h):
    g = torch.Generator(device="cuda").manual_seed(k + h)
    hq = h * group
    q = torch.randn((R, hq, 128), generator=g, device="cuda").mul(0.5).to(torch.bfloat16)
    rows = marked(k, h, 16, g).repeat(R, 1)
    # the places of all requests' rows in the cache, in no order
    place = torch.randperm(R * k, generator=g, device="cuda")
    cache = torch.empty_like(rows)
    cache[place] = rows
    idx = place.view(R, k).to(torch.int32)
    out = prefix_attention(q, None, 0, cache, R * k, idx, R, k, hq, h)
    for r in sorted({0, R // 3, R - 1}):
        check(q[r], rows[:k], out[r], h, 16)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("h,group", [(8, 1), (4, 4), (2, 16)])
def test_probabilities_of_published_rows_keep_two_terms(h, group, weights):
    """Two kinds of rows whose values nearly cancel, +1 against minus the bf16
    nearest their ratio of weights: what is left is what a single rounding of the
    probabilities to bf16 would lose."""
    hq, k = h * group, 200
    # of each query: score 0 to the first kind of row, -x to the second
    x = torch.linspace(0.03, 0.65, hq, device="cuda", dtype=torch.float64)
    q = torch.zeros((1, hq, 128), device="cuda")
    q[0, :, 0] = -(x / SCALE).float()
    q = q.to(torch.bfloat16)
    ratio = torch.exp(q[0, :, 0].double() * SCALE)          # the second kind's weight
    cache = torch.zeros((k, 2, h, 128), device="cuda")
    cache[1::2, 0, :, 0] = 1.0
    # dimension j of a head: cancels for its j-th query
    near = ratio.float().to(torch.bfloat16).float().view(h, group)
    cache[0::2, 1, :, :group] = -near
    cache[1::2, 1, :, :group] = 1.0
    cache = cache.to(torch.bfloat16).view(k, h * 256)
    idx = torch.randperm(k, device="cuda").to(torch.int32)[None].contiguous()
    if weights:
        out = torch.empty((1, hq, 128), dtype=torch.bfloat16, device="cuda")
        need = hs.hs_attention_weights_bytes(1, hq, h, k)
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        acc = torch.zeros((1, k), device="cuda")
        hs.hs_sparse_attention_weights(q, cache, k, idx, idx, 1, k, hq, h, SCALE, out, acc, 1, k, work,
                                       need)
    else:
        out = prefix_attention(q, None, 0, cache, k, idx, 1, k, hq, h)
    keys, values = ref.split(cache, h)
    want, p, _, rel = ref.attention(q[0], keys, values, SCALE)
    mass = torch.einsum("hgn,hnd->hgd", p.view(h, group, k), values.abs()).reshape(hq, 128)
    # as the bound of ref.attention, with 2^-17 for the two terms of a probability
    bound = mass * (2.0 ** -17 + rel + k * 2.0 ** -23) + ref.BF16 * want.abs() * (1 + ref.BF16)
    assert bool(((out[0].double() - want).abs() <= bound).all())
    # the same with one term (relative to the largest, as the probabilities are
    # held): outside the bound for most queries, so the bound can tell
    one = torch.stack((torch.ones_like(ratio), ratio.float().to(torch.bfloat16).double()), 1)
    one = (one / (1 + ratio)[:, None] / (k // 2)).repeat(1, k // 2).view(h, group, k)
    lost = (torch.einsum("hgn,hnd->hgd", one, values).reshape(hq, 128) - want).abs() > bound
    assert lost.any(1).double().mean().item() > 0.7

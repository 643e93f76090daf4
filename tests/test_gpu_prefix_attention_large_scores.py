"""hs_prefix_attention where scores are so large that one key takes all the
weight: the softmax is one at the largest score and the output is that key's
value, for scores from some thousands to 2^60."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** 6, 2.0 ** 10, 2.0 ** 14, 2.0 ** 17, 2.0 ** 20, 2.0 ** 30])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("R,P,k,hq,h", [
    (2, 40, 0, 4, 4), (3, 700, 20, 8, 2), (9, 5000, 0, 28, 7), (60, 900, 33, 16, 4), (300, 3000, 5, 8, 8)])
def test_the_largest_score_takes_all(R, P, k, hq, h, sign, size):
    g = torch.Generator(device="cuda").manual_seed(P + k)

    def bf16(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    rows = max(1, R * k)
    q, prefix, cache = bf16(R, hq, 128, scale=size), bf16(P, h * 256), bf16(rows, h * 256)
    prefix[:, :h * 128] *= size
    cache[:, :h * 128] *= size
    idx = torch.arange(R * k, device="cuda", dtype=torch.int32).view(R, k)
    out = torch.empty((R, hq, 128), dtype=torch.bfloat16, device="cuda")
    need = hs.hs_prefix_attention_bytes(R, hq, h, P, k)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    scale = sign * 128 ** -0.5
    hs.hs_prefix_attention(q, prefix, P, cache, rows, idx, R, k, hq, h, scale, out, work, need)
    qg = q.double().view(R, h, hq // h, 128)
    keys, values = prefix.view(P, 2, h, 128).transpose(0, 1)
    s = torch.einsum("rhgd,phd->rhgp", qg, keys.double()) * scale
    values = values.permute(1, 0, 2).expand(R, h, P, 128)
    if k:
        own = cache.view(R, k, 2, h, 128)
        s = torch.cat((s, torch.einsum("rhgd,rphd->rhgp", qg, own[:, :, 0].double()) * scale), -1)
        values = torch.cat((values, own[:, :, 1].permute(0, 2, 1, 3)), 2)
    top, at = s.topk(2, -1)
    # a score is off by at most 2^-16 of the sum of its products' magnitudes (128
    # additions of 2^-23 each), below 2^-16 * 128 * (6 size)^2 * |scale|; where the
    # two largest are further apart than twice that and 40, all the other weights
    # are below 5033 e^-40 < 2^-44 in sum
    off = 2.0 ** -16 * 128 * 36 * size * size * abs(scale)
    sure = top[..., 0] - top[..., 1] > 2 * off + 40
    assert bool(sure.any())
    want = torch.gather(values, 2, at[..., :1].expand(R, h, hq // h, 128))
    got = out.view(R, h, hq // h, 128)
    assert not bool(got.isnan().any())
    # the value times its probability, which is rounded once to bf16 before the
    # sum divides it; the result rounded once; the other values (below 8)
    got, want = got[sure].double(), want[sure].double()
    assert bool(((got - want).abs() <= want.abs() * (2.0 ** -7 + 2.0 ** -15) + 2.0 ** -40).all())

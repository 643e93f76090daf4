"""hs_packed_attention with queries and rows whose products and sums fp32 holds
exactly, so that the bound on the output is a few roundings wide however large the
scores are; and large queries, where one row takes all the weight."""
import math

import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import latent_reference as ref
from tests.test_gpu_packed_attention import SCALE, attend, make

pytestmark = pytest.mark.gpu
P_REL = torch.finfo(torch.float16).eps / 2   # half a step of f16: 2^-11
P_ABS = 2.0 ** -32                           # half of f16's least step, in units of 2^-7 of a probability


def exact(R, k, h, seed):
    """Rows of e2m1 values with scale 1 and small whole numbers beside them, queries
    of whole numbers up to 8: every product is a multiple of 1/2, every sum below
    576 * 8 * 6 = 27648 -- 16 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = R * k + 5

    def whole(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(torch.bfloat16)

    level = torch.tensor(ref.E2M1 + [-x for x in ref.E2M1], device="cuda")
    x = level[torch.randint(0, 16, (rows, 576), generator=g, device="cuda")]
    x[:, 0:512:16] = 6.0
    x[:, 512:] = whole(4, rows, 64)
    x = x.to(torch.bfloat16)
    cache = ref.pack(x, 0)
    assert torch.equal(ref.values(cache, 0), x.double())
    return dict(R=R, k=k, h=h, q=whole(8, R, h, 576), rows=rows, g=g, shift=0, cache=cache,
                idx=torch.randperm(rows, generator=g, device="cuda")[:R * k].view(R, k).to(torch.int32).contiguous())


# Scores s = acc * (scale * log2 e * 2^j): acc exact, the factor off by 2 * 2^-24 (the
# constant, its product with the scale), one more for the product: 3 * 2^-24 of S, the
# largest; base and difference 2 * 2^-24 of at most 2 S.  As exponents they make a
# probability wrong by 7 * 2^-24 S, and ex2 by 2^-22; in the sum once more.  A rise
# multiplies what is there by ex2(difference of two bases): 2^-22 and 4 * 2^-24 S, at
# most once a tile, and once more where parts are joined.
def definition(s, r, scale):
    keys = ref.values(s["cache"][s["idx"][r].long()], 0)
    q = s["q"][r].double()
    scores = q @ keys.T * scale
    top, n = scores.abs().max().item(), keys.shape[0]
    p = torch.softmax(scores, -1)
    out, weight = p @ keys[:, :512], p @ keys[:, :512].abs()
    tiles = -(-n // 128)
    rel = 2 * (7 * 2.0 ** -24 * top + 2.0 ** -22) + (tiles + 1) * (2.0 ** -22 + 4 * 2.0 ** -24 * top)
    # the sum and the output: n additions each
    return out, weight * (P_REL * 2 + rel + 2 * n * 2.0 ** -24) + P_ABS * 2 * keys[:, :512].abs().sum(0) + \
        ref.BF16 * out.abs() * (1 + ref.BF16)


# the scores' deviation is sqrt(576) * 4.9 * 2.7 * scale: from 3 nats to 300
@pytest.mark.parametrize("scale", [0.01, -0.03, 0.1, 0.3, 1.0])
@pytest.mark.parametrize("R,k,h", [(3, 333, 5), (2, 1000, 16), (2, 600, 33), (2, 777, 64), (1, 2048, 128)])
def test_exact_scores(R, k, h, scale):
    s = exact(R, k, h, k + h)
    out = attend(s, scale=scale)
    for r in range(R):
        want, bound = definition(s, r, scale)
        assert bool((bound.amax(-1) < want.abs().amax(-1) / 8).all())      # a bound that zeros would miss
        err = (out[r].double() - want).abs()
        assert bool((err <= bound).all()), (r, (err - bound).max().item(), err.max().item())


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_exact_scores_in_order(order):
    s = exact(4, 1300, 40, 9)
    keys = ref.values(s["cache"], 0)
    for r, head in enumerate((0, 13, 31, 39)):
        by = (keys[s["idx"][r].long()] @ s["q"][r, head].double()).argsort(descending=order == "falling")
        s["idx"][r] = s["idx"][r][by]
    out = attend(s, scale=0.2)
    for r in range(4):
        want, bound = definition(s, r, 0.2)
        assert bool(((out[r].double() - want).abs() <= bound).all()), r


@pytest.mark.parametrize("h", [5, 16, 64])
@pytest.mark.parametrize("q_scale", [300.0, 1e6, 1e20])
def test_one_row_takes_all_the_weight(q_scale, h):
    """Where the first score leads by 40 nats more than two scores can be off, the
    output is that row's values, rounded once; what is left for the others is below
    k e^-40."""
    s = make(4, 150, h, h)
    s["q"] = (s["q"].double() * q_scale).to(torch.bfloat16)
    out = attend(s)
    for r in range(4):
        keys = ref.values(s["cache"][s["idx"][r].long()], 0)
        q = s["q"][r].double()
        two = (q @ keys.T * SCALE).topk(2)
        off = (q.abs() @ keys.abs().T).amax(-1) * SCALE * (576 * 2.0 ** -23 + 4 * 2.0 ** -24)
        clear = two.values[:, 0] - two.values[:, 1] > 40 + 2 * off
        assert int(clear.sum()) >= h // 4 + 1
        want = keys[two.indices[:, 0], :512]
        bound = ref.BF16 * want.abs() + 150 * math.exp(-40) * keys[:, :512].abs().amax()
        assert bool(((out[r].double() - want).abs() <= bound)[clear].all())
    assert hs.hs_attention_status() == 0

"""hs_latent_prefill where a pair's keys are split among CTAs and one part holds
next to none of a query's weight: an infinity or NaN among the values that the
query sees shows all the same, as it does where nothing is split."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests.test_gpu_latent_prefill import attend, make

pytestmark = pytest.mark.gpu


def light(n, m, h, heavy):
    """Keys `heavy` take all the weight of every query: their scores pass the others'
    by about 30 * 100 / sqrt(192) = 216 nats, more than fp32's exponents hold."""
    s = make([n], [m], h, n + m)
    s["q"][:, :, 0] = 30
    s["kv"][:, :, 0] = 0
    s["kv"][heavy, :, 0] = 100
    return s


# of 12000 keys the first 9000 are in one part or more of their own; the heavy ones
# come later, and are seen by every query (or, the other way round, before them)
@pytest.mark.parametrize("n,m,h,heavy,key", [(300, 12000, 64, slice(11600, 11650), 5), (100, 9000, 8, slice(8800, 8850), 3),
                                             (300, 12000, 64, slice(0, 50), 11600), (100, 9000, 8, slice(0, 50), 8880)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_light_parts_keep_infinities_and_nan(n, m, h, heavy, key, bad):
    assert hs.hs_latent_prefill_bytes(n, m, 1, h) > 0           # split
    s = light(n, m, h, heavy)
    want = attend(s)
    assert bool(torch.isfinite(want).all())
    s["kv"][key, 3, 128 + 77] = bad
    out = attend(s)
    got = out[:, 3, 77].float()
    assert bool((torch.isnan(got) if bad != bad else ~torch.isfinite(got)).all())
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:, 3, 77] = True
    assert torch.equal(out[~hit].view(torch.int16), want[~hit].view(torch.int16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_and_so_does_an_unsplit_call(bad):
    s = light(2, 256, 2, slice(200, 250))
    s["kv"][5, 1, 128 + 77] = bad
    assert hs.hs_latent_prefill_bytes(2, 256, 1, 2) == 0
    assert not bool(torch.isfinite(attend(s)[:, 1, 77].float()).any())


def test_light_parts_weigh_nothing_else():
    """Large finite values of a part without weight add nothing."""
    s = light(300, 12000, 64, slice(11600, 11650))
    want = attend(s)
    s["kv"][:9000, :, 128:] = 1e30
    assert torch.equal(attend(s).view(torch.int16), want.view(torch.int16))

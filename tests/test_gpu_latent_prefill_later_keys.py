"""hs_latent_prefill: a key that a query does not see changes no bit of its output,
large finite keys among them, which move the maxima of the queries that do see
them."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests.test_gpu_latent_prefill import attend, check, make

pytestmark = pytest.mark.gpu


def bits(x):
    return x.contiguous().view(torch.int16)


def enlarge(s, key, query, factor):
    """The key becomes `factor` times the query that first sees it: its score passes
    the others' of that query by |q|^2 factor SCALE, about 21 factor nats."""
    s["kv"][key, :, :128] = s["q"][query, :, :128] * factor


@pytest.mark.parametrize("factor", [1.0, 16.0, 2.0 ** 22])
@pytest.mark.parametrize("n,m,at", [(400, 450, 1), (400, 450, 90), (400, 450, 100), (400, 450, 130), (400, 450, 255),
                                    (400, 450, 399), (257, 1257, 30), (64, 20000, 31), (300, 12000, 40)])
def test_large_keys_leave_earlier_queries_as_they_were(n, m, at, factor):
    s = make([n], [m], 8, n + at)
    want = attend(s)
    enlarge(s, m - n + at, at, factor)
    out = attend(s)
    assert torch.equal(bits(out[:at]), bits(want[:at]))
    assert not torch.equal(bits(out[at]), bits(want[at]))


def test_prompts_that_go_on_differently():
    """Two prompts alike up to some token give that part alike, whatever follows."""
    s = make([513], [700], 4, 3)
    want = attend(s)
    for at in (7, 40, 77, 129, 200, 300, 511):
        t = {**s, "kv": s["kv"].clone(), "rec": s["rec"].clone()}
        t["kv"][187 + at:] = t["kv"][187 + at:].flip(0) * 32
        t["rec"][187 + at:] = t["rec"][187 + at:].flip(0) * 32
        assert torch.equal(bits(attend(t)[:at]), bits(want[:at])), at


def test_maxima_that_rise_for_some_queries_only():
    """Keys that single queries score high with, in every block."""
    s = make([300], [900], 3, 5)
    for i in range(0, 300, 11):
        enlarge(s, (i * 37) % 600, i, 1.0)
    out = attend(s)
    check(s, out)
    assert torch.equal(bits(out), bits(attend(s)))


@pytest.mark.parametrize("lens,keys", [([1], [9000]), ([257], [257]), ([300, 129, 5], [700, 129, 2000]),
                                       ([40, 30], [1000, 0]), ([700, 300], [500, 299])])
def test_rows_behind_a_sequence_and_queries_that_see_nothing(lens, keys):
    """Tiles with rows that see no key, over several blocks."""
    s = make(lens, keys, 4, sum(lens))
    for i in range(0, sum(keys), 50):
        s["kv"][i, :, :128] *= 3
    out = attend(s)
    check(s, out)
    for i, (n, m) in enumerate(zip(lens, keys)):
        if n > m:
            assert bool((out[sum(lens[:i]):sum(lens[:i]) + n - m] == 0).all())
    assert hs.hs_attention_status() == 0

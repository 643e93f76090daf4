"""The angles of hs_qk_norm_rope at far positions and for frequencies of any
size, against exact rational arithmetic (a double's product of the two has lost
them long before)."""
from fractions import Fraction

import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref

pytestmark = pytest.mark.gpu
# 64 digits: exact to 1e-64, and 2^31 * 2^55 radians are below 1e27
TURN = 2 * Fraction("3.1415926535897932384626433832795028841971693993751058209749445923")


def angle(pos, freq):
    """pos * freq modulo one turn, in (-pi, pi], as a double."""
    t = Fraction(pos) * Fraction(freq) / TURN
    t -= round(t)
    return float(t * TURN)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("freqs", [
    [10000.0 ** (-i / 64) for i in range(64)], [-10000.0 ** (-i / 16) for i in range(16)],
    [3.7, 41.0, -977.0, 1e5 / 3, -1e6 / 7, 1e7 / 9, 1e8 / 11, 1e9 / 13],
    [1e10 / 17, -1e11 / 19, 1e12 / 23, 1e14 / 29, -1e15 / 31, 3.3e16, -5.5e16, 2.0 ** 55],
    [1e-9, -1e-9, 1e-12, -1e-15, -1e-18, 2.0 ** -62, -2.0 ** -62, -1e-300]])
def test_angles_at_any_position_and_frequency(freqs, inter):
    n, hq, h = 6, 3, 2
    g = torch.Generator(device="cuda").manual_seed(len(freqs))
    q, k, v = (torch.randn((n, x, 128), generator=g, device="cuda").to(torch.bfloat16)
               for x in (hq, h, h))
    where = [1, -12345, 999983, 123456789, (1 << 31) - 1, -(1 << 31)]
    pos = torch.tensor(where, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(q)
    records = torch.empty((n, 2 * h, 128), dtype=torch.bfloat16, device="cuda")
    hs.hs_qk_norm_rope(hs.qk_desc(hq, h, freqs, interleaved=inter), q, k, v, None, None, pos, n, q_out,
                       records, n)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    for i, p in enumerate(where):
        turned = [angle(p, f) for f in freqs]
        for got, x in ((q_out[i:i + 1], q[i:i + 1]), (records[i:i + 1, :h], k[i:i + 1])):
            y, size = ref.norm_rope(x, None, one, turned, 1e-6, inter)
            # the bound covers pi * 2^-24 of the angle (its own part allows 2^-21)
            err = (got.double() - y).abs()
            assert bool((err <= ref.norm_rope_bound(y, size)).all()), (p, err.max().item())

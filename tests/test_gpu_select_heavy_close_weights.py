"""hs_select_heavy on weights that lie close together, as nearly flat attention
accumulates them: the border falls among many equal weights with others a few
units in the last place above them, at every width of the bins in which the
border is sought, and at every number of blocks that share a request.  Exact,
against a stable sort; the selection is filled with a mark beforehand, so that
a place that is left out shows."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs

pytestmark = pytest.mark.gpu

# requests and positions for which 1, 2, 4, 8, 12 and 16 blocks share a request
SHAPES = [(80, 4000), (40, 4100), (20, 8300), (9, 16500), (8, 24700), (3, 33000)]


def check(w, k, recent):
    """w [n][L] fp32 on the host."""
    n, L = w.shape
    sel = torch.full((n, k), -9, dtype=torch.int32, device="cuda")
    hs.hs_select_heavy(w.cuda(), n, L, None, n, k, recent, sel)
    got = sel.cpu()
    last = min(recent, L)
    for i in range(n):
        order = torch.sort(w[i, :L - last].double(), descending=True, stable=True).indices
        kept = sorted(order[:k - last].tolist()) + list(range(L - last, L))
        assert got[i].tolist() == kept + [-1] * (k - len(kept)), i


def weight_of(key):
    """The weights whose unsigned order numbers are `key` (int64)."""
    bits = torch.where(key >= 1 << 31, key - (1 << 31), (1 << 32) - 1 - key)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).view(torch.float32)


@pytest.mark.parametrize("n,L", SHAPES)
@pytest.mark.parametrize("equal", [33, 100])
def test_equal_weights_at_the_border_under_close_ones(n, L, equal):
    """`equal` weights one unit above a multiple of 2^21 (in the weights' order,
    where a first bound lies), 60 others up to 2047 units higher, and one 2^e
    units higher, which sets the width of the bins: for every e."""
    g = torch.Generator().manual_seed(L + equal)
    cases = []
    for e in range(11, 32):
        # a base with room for 2^e above it: 1.0, the smallest normal weights, or
        # negative ones
        base = 0xBF800000 if e <= 29 else 0x80800000 if e == 30 else 0x7F000000
        keys = torch.cat((torch.full((equal,), base + 1, dtype=torch.int64),
                          base + torch.randint(2, 2048, (60,), generator=g),
                          torch.tensor([base + (1 << e) + (1 << e) // 7])))
        if e == 31:
            keys[-1] = 0xFF000000           # (finite, more than 2^31 above the base)
        row = torch.full((L,), 0.0 if e < 31 else -3e38)
        row[torch.randperm(L, generator=g)[:keys.numel()]] = weight_of(keys)
        assert bool(row.isfinite().all())
        cases.append(row)
    # 61 above the equal ones, then about half of those
    for at in range(0, len(cases), n):
        some = cases[at:at + n]
        while len(some) < n:
            some.append(cases[len(some) % len(cases)])
        check(torch.stack(some), 61 + equal // 2, 0)


@pytest.mark.parametrize("n,L", SHAPES)
def test_clusters_of_close_weights_at_several_heights(n, L):
    """Three clusters of weights within 2047 units of one another, 2^12 to 2^22
    units apart, under one far above; the border in each."""
    g = torch.Generator().manual_seed(L)
    rows = []
    for i in range(n):
        apart = 1 << 12 + i % 11
        base = 0x3F800000 + torch.tensor([0, apart, 3 * apart])
        keys = torch.cat([b + torch.randint(0, 2048, (150,), generator=g) // 40 * 40 for b in base])
        row = torch.zeros(L, dtype=torch.int32)
        place = torch.randperm(L, generator=g)[:keys.numel() + 1]
        row[place[:-1]] = keys.to(torch.int32)
        row[place[-1]] = 0x41200000         # 10.0
        rows.append(row.view(torch.float32))
    w = torch.stack(rows)
    for k in (40, 151, 200, 299, 330, 440):
        check(w, k, 0)


@pytest.mark.parametrize("n,L", SHAPES)
@pytest.mark.parametrize("spread", [1e-6, 1e-5, 3e-5, 1e-4, 1e-3, 1e-2])
def test_nearly_flat_weights(n, L, spread):
    """w (1 + spread N(0, 1)), alone and beside one position that draws 1.2, 10
    and 10^4 times as much."""
    g = torch.Generator().manual_seed(int(L * spread * 1e6))
    w = 1.05 * (1 + spread * torch.randn((n, L), generator=g))
    for i, sink in enumerate((1.0, 1.2, 10.0, 1e4)):
        w[i::4, 3 * i] *= sink
    for k, recent in ((50, 0), (600, 8), (2048, 64)):
        check(w, k, recent)

"""hs_select_heavy against a plain sort, exactly: lengths from none to long,
ties, zeros of both signs, infinities and NaN, request ids, short requests,
and the largest and smallest counts."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref

pytestmark = pytest.mark.gpu


def select(w, lens, k, recent, ids=None, n_req=None, stream=None):
    n = w.shape[0] if n_req is None else n_req
    sel = torch.full((n, k), -9, dtype=torch.int32, device="cuda")
    hs.hs_select_heavy(w, w.shape[0], w.shape[1], lens, n, k, recent, sel, ids, stream)
    return sel


def want(w, lens, k, recent, ids=None):
    """The same by a stable sort on the host."""
    out = []
    for i in range(len(lens)):
        req = i if ids is None else ids[i]
        if not 0 <= req < w.shape[0]:
            out.append([-1] * k)
            continue
        n = min(max(lens[i], 0), w.shape[1])
        last = min(recent, n)
        v = w[req, :n - last].cpu().double()
        v = torch.where(v.isnan(), -float("inf"), v)
        order = torch.sort(v, descending=True, stable=True).indices[:k - last]
        kept = sorted(order.tolist()) + list(range(n - last, n))
        out.append(kept + [-1] * (k - len(kept)))
    return torch.tensor(out, dtype=torch.int32)


def heavy_tailed(n, L, seed, zeros=0.4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.exp(2.5 * torch.randn((n, L), generator=g, device="cuda") - 6)
    w[torch.rand((n, L), generator=g, device="cuda") < zeros] = 0
    return w


@pytest.mark.parametrize("n,L,k,recent", [
    (1, 1, 1, 0), (1, 1, 1, 1), (2, 5, 3, 1), (3, 100, 10, 4), (3, 1023, 64, 16), (4, 1024, 64, 64),
    (4, 1025, 200, 0), (32, 4096, 2048, 64), (5, 20000, 777, 33), (2, 131072, 2048, 64),
    (7, 99991, 4096, 256), (1, 1048576, 2048, 64), (3, 1 << 20, 1, 0), (70, 3000, 100, 10)])
def test_against_a_sort(n, L, k, recent):
    w = heavy_tailed(n, L, n + L)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = torch.randint(L // 2, L + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = L
    assert torch.equal(select(w, lens, k, recent).cpu(), want(w, lens.tolist(), k, recent))
    assert torch.equal(select(w, None, k, recent).cpu(), want(w, [L] * n, k, recent))


def test_agrees_with_the_list_reference():
    w = heavy_tailed(2, 300, 4)
    got = select(w, None, 50, 7).cpu().tolist()
    for r in range(2):
        assert got[r] == ref.keep(w[r].tolist(), 300, 50, 7)


@pytest.mark.parametrize("k,recent", [(64, 0), (64, 8), (64, 64), (500, 3)])
def test_short_and_out_of_range_lengths(k, recent):
    L = 400
    lens = [0, 1, recent, recent + 1, k - 1, k, k + 1, L - 1, L, L + 5, -3]
    w = heavy_tailed(len(lens), L, 9)
    d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert torch.equal(select(w, d, k, recent).cpu(), want(w, lens, k, recent))


def test_ties_go_to_the_lowest_position():
    L, k = 70000, 1000
    w = torch.zeros((4, L), device="cuda")
    w[1] = 0.25
    w[2, ::7] = 1.0                      # 10000 equal maxima
    w[3, ::100] = 2.0                    # 700 maxima, then zeros
    w[3, 1::2] *= -1                     # among them -0
    lens = [L] * 4
    assert torch.equal(select(w, None, k, 10).cpu(), want(w, lens, k, 10))
    assert select(w, None, k, 0)[0].tolist() == list(range(k))


def test_negative_infinite_and_nan_weights():
    L, k = 3000, 256
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn((5, L), generator=g, device="cuda")
    w[0] = -w[0].abs()
    w[1, ::3] = float("inf")
    w[2, ::2] = -float("inf")
    w[2, 1::4] = float("nan")
    w[3] = float("nan")
    w[4] *= 1e-42                         # denormals
    w[4, 5] = -1e-45
    assert torch.equal(select(w, None, k, 16).cpu(), want(w, [L] * 5, k, 16))


def test_keys_that_differ_only_in_their_last_bits():
    """Weights of consecutive floats: every bit of the key decides."""
    L, k = 5000, 333
    g = torch.Generator(device="cuda").manual_seed(3)
    base = torch.tensor([0.75], device="cuda").view(torch.int32)
    w = (base + torch.randperm(L, generator=g, device="cuda").to(torch.int32)).view(torch.float32)[None]
    assert torch.equal(select(w, None, k, 5).cpu(), want(w, [L], k, 5))


@pytest.mark.parametrize("n,L,k", [(1, 131072, 4096), (2, 60000, 3000), (9, 300000, 2500), (80, 9000, 700)])
def test_heavy_positions_all_in_one_place(n, L, k):
    """The heaviest positions next to one another: one CTA's share of the
    candidates holds all of them."""
    w = torch.linspace(1.0, 0.5, L, device="cuda").repeat(n, 1).contiguous()
    assert torch.equal(select(w, None, k, 8).cpu(), want(w, [L] * n, k, 8))
    w = w.flip(1).contiguous()
    assert torch.equal(select(w, None, k, 8).cpu(), want(w, [L] * n, k, 8))


@pytest.mark.parametrize("n,L,k", [(80, 200001, 2000), (80, 400003, 300), (2, 1 << 23, 4000), (77, 70000, 5000)])
def test_long_ranges_of_one_block(n, L, k):
    """Many positions to each block: one block to a request, or several with
    half a million each; heavy positions only here and there, in the first and
    the last places among them."""
    w = heavy_tailed(n, L, L + k)
    w[:, 0], w[:, -9], w[:, L // 2] = 900.0, 901.0, 900.0
    w[1, L // 3:2 * L // 3] = 0
    assert torch.equal(select(w, None, k, 8).cpu(), want(w, [L] * n, k, 8))


def test_many_equal_weights_at_the_border():
    """More equal weights than any list holds, on both sides of the border, and
    long rows of NaN and -infinity."""
    L, k = 200000, 1500
    w = torch.full((5, L), 0.5, device="cuda")
    w[1, ::300] = 0.75                    # 667 above, the rest equal
    w[2, 1::2] = 0.500001                 # 100000 equal, above 100000 others
    w[3] = float("nan")
    w[4] = -float("inf")
    w[4, ::1000] = -1e30
    assert torch.equal(select(w, None, k, 16).cpu(), want(w, [L] * 5, k, 16))


def test_request_ids():
    w = heavy_tailed(6, 2000, 11)
    ids = [5, 0, -1, 6, 3, 3]
    lens = [1500, 2000, 100, 2000, 700, 2000]
    got = select(w, torch.tensor(lens, dtype=torch.int32, device="cuda"), 128, 32,
                 torch.tensor(ids, dtype=torch.int32, device="cuda"), n_req=6)
    assert torch.equal(got.cpu(), want(w, lens, 128, 32, ids))


def test_a_large_k_and_one_past_the_context():
    w = heavy_tailed(2, 30000, 12)
    for k in (29999, 30000, 30001, 32767):
        assert torch.equal(select(w, None, k, 100).cpu(), want(w, [30000] * 2, k, 100))


def test_graph_replay_and_side_stream():
    w = heavy_tailed(4, 9000, 13)
    lens = torch.full((4,), 9000, dtype=torch.int32, device="cuda")
    sel = torch.zeros((4, 200), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = select(w, lens, 200, 8, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want(w, [9000] * 4, 200, 8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_select_heavy(w, 4, 9000, lens, 4, 200, 8, sel)
    w.copy_(heavy_tailed(4, 9000, 14))
    lens -= 77
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(sel.cpu(), want(w, [8923] * 4, 200, 8))


def test_unaligned_rows_and_guards():
    """n_positions that is no multiple of four: rows start at any 4-byte
    boundary; nothing is written outside the selection."""
    L, k = 1003, 50
    big = heavy_tailed(1, 5 * L + 1, 15)[0]
    w = big[1:].view(5, L)
    buf = torch.full((5 * k + 64,), -9, dtype=torch.int32, device="cuda")
    hs.hs_select_heavy(w, 5, L, None, 5, k, 3, buf[32:])
    torch.cuda.synchronize()
    assert torch.equal(buf[32:32 + 5 * k].view(5, k).cpu(), want(w, [L] * 5, k, 3))
    assert bool((buf[:32] == -9).all()) and bool((buf[32 + 5 * k:] == -9).all())


def test_refusals():
    w = heavy_tailed(1, 100, 16)
    with pytest.raises(hs.HsError) as e:
        select(w, None, 10, 11)
    assert e.value.code == hs.HS_ERR_INVALID_ARG

"""hs_prefix_attention against its definition in 64 bits (tests/token_reference.py,
where the bound is derived): prefix lengths and own selections around the tile
sizes, group sizes 1 to 16, head counts 1 to 8, batches that fill part of a
tile and several tiles, masked rows, no rows, no prefix, infinities in masked
places, repeated calls, other streams and captured graphs."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def bf16(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def make(R, P, k, hq, h, seed, q_scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = R * k + 5
    return dict(R=R, P=P, k=k, hq=hq, h=h, q=bf16(g, R, hq, 128, scale=q_scale),
                prefix=bf16(g, P, h * 256) if P else None, rows=rows, cache=bf16(g, rows, h * 256),
                idx=torch.randperm(rows, generator=g, device="cuda")[:R * k].view(R, k)
                .to(torch.int32).contiguous(), g=g)


def attend(s, out=None, work=None, stream=None, scale=SCALE, **kw):
    s = {**s, **kw}
    if out is None:
        out = torch.full((s["R"], s["hq"], 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    need = hs.hs_prefix_attention_bytes(s["R"], s["hq"], s["h"], s["P"], s["k"])
    if work is None:
        work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    hs.hs_prefix_attention(s["q"], s["prefix"], s["P"], s["cache"], s["rows"], s["idx"], s["R"],
                           s["k"], s["hq"], s["h"], scale, out, work, need, stream)
    return out


def check(s, out, scale=SCALE, requests=None):
    for r in requests if requests is not None else range(s["R"]):
        rows = s["prefix"][:s["P"]] if s["P"] else s["cache"][:0]
        if s["k"]:
            idx = s["idx"][r].long()
            own = s["cache"][idx[(idx >= 0) & (idx < s["rows"])]]
            rows = torch.cat((rows, own)) if s["P"] else own
        keys, values = ref.split(rows, s["h"])
        want, _, bound, _ = ref.attention(s["q"][r], keys, values, scale)
        err = (out[r].double() - want).abs()
        assert bool((err <= bound).all()), (r, (err - bound).max().item(), err.max().item())


@pytest.mark.parametrize("R,P,k,hq,h", [
    (1, 1, 0, 1, 1), (1, 1, 1, 8, 8), (2, 517, 33, 8, 8), (3, 127, 0, 4, 4), (3, 128, 5, 8, 2),
    (3, 129, 64, 16, 1), (5, 255, 65, 15, 5), (5, 257, 128, 21, 3), (2, 1000, 1000, 28, 7),
    (7, 4096, 100, 48, 6), (19, 20011, 0, 12, 4), (33, 3000, 40, 32, 8), (64, 1500, 17, 64, 8),
    (65, 700, 3, 16, 4), (130, 640, 31, 8, 8), (300, 384, 9, 3, 1), (40, 2500, 200, 128, 8)])
def test_against_definition(R, P, k, hq, h):
    s = make(R, P, k, hq, h, R * 1000 + P + k)
    out = attend(s)
    again = attend(s)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    check(s, out, requests=sorted({0, 1 % R, R // 2, R - 1}))


@pytest.mark.parametrize("k", [1, 15, 16, 17, 31, 32, 33, 100, 511, 2048, 5000])
def test_own_rows_alone(k):
    s = make(3, 0, k, 24, 8, k)
    out = attend(s)
    check(s, out)


@pytest.mark.parametrize("P", [0, 300])
@pytest.mark.parametrize("h", [1, 2, 3, 4, 5, 6, 7, 8])
def test_long_selections_of_every_record_size(h, P):
    """Ranges of rows many times as long as the ring that brings them, requests
    that end inside a range, one row in five masked, one request without any."""
    s = make(30, P, 4001, 3 * h, h, 500 + h)
    s["idx"][torch.rand(s["idx"].shape, generator=s["g"], device="cuda") < 0.2] = -1
    s["idx"][17] = s["rows"]
    out = attend(s)
    check(s, out, requests=[0, 1, 16, 18, 29] + ([17] if P else []))
    if not P:
        assert bool((out[17] == 0).all())
    for _ in range(5):
        assert torch.equal(attend(s).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("h", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 11, 16])
def test_head_layouts(h, group):
    s = make(3, 300, 70, h * group, h, h * 100 + group)
    check(s, attend(s))


@pytest.mark.parametrize("R,hq,h,P,k", [
    (48, 8, 1, 5000, 100),      # 384 queries to one head: a pair of tiles and half a pair
    (100, 32, 8, 1000, 5),      # 400 to each of eight heads
    (700, 16, 1, 900, 2),       # 11200 queries: 44 pairs of tiles
    (2500, 128, 8, 300, 1),     # 40000 to each head: more pairs of tiles than SMs
    (9, 112, 7, 30000, 300)])   # ranges of the prefix that reach into a second head
def test_many_tiles_and_ranges(R, hq, h, P, k):
    s = make(R, P, k, hq, h, R + P)
    check(s, attend(s), requests=sorted({0, 1, R // 3, R // 2, R - 2, R - 1}))


@pytest.mark.parametrize("R,hq,P,k", [(9, 56, 50000, 0), (18, 49, 60000, 40), (1, 112, 47001, 3)])
def test_one_tile_of_queries_and_ranges_into_a_second_head(R, hq, P, k):
    """Up to 128 queries to each of seven heads, which do not divide the SMs:
    many ranges of the prefix end in another head than they start in, where the
    next head's queries take the place of the last one's."""
    s = make(R, P, k, hq, 7, P)
    out = attend(s)
    check(s, out, requests=sorted({0, R // 2, R - 1}))
    for _ in range(20):
        assert torch.equal(attend(s).view(torch.int16), out.view(torch.int16))


def test_a_request_for_every_place_of_a_tile():
    """Groups that do not divide a tile of rows: requests straddle tiles."""
    for hq, R in ((5, 60), (7, 40), (3, 100), (11, 50), (13, 30)):
        s = make(R, 260, 6, hq, 1, hq)
        check(s, attend(s))


def test_masked_rows_and_requests_without_rows():
    s = make(6, 0, 150, 16, 8, 77)
    s["idx"][0] = -1
    s["idx"][1, ::3] = s["rows"]
    s["idx"][2, 1:] = -1
    s["idx"][3, :64] = -5
    s["idx"][4, 64:] = 1 << 30
    out = attend(s)
    assert bool((out[0] == 0).all())
    check(s, out, requests=range(1, 6))
    s2 = make(6, 90, 150, 16, 8, 78)
    s2["idx"] = s["idx"].clone()
    s2["rows"] = s["rows"]
    out = attend(s2)
    check(s2, out)


def test_no_rows_at_all():
    s = make(3, 0, 0, 8, 4, 1)
    out = attend(s, cache=None, idx=None, rows=0)
    assert bool((out == 0).all())


def test_rows_outside_the_prefix_and_the_selection_are_never_used():
    """NaN and infinity in the cache rows that no valid index names, in the
    row behind the prefix, and at the masked indices' place."""
    R, P, k, hq, h = 4, 200, 40, 16, 4
    s = make(R, P, k, hq, h, 55)
    big = torch.full((P + 300, h * 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:P] = s["prefix"]
    s["prefix"] = big                     # the same prefix, NaN behind it
    s["idx"][:, 7] = -1
    used = torch.zeros(s["rows"], dtype=torch.bool, device="cuda")
    used[s["idx"][s["idx"] >= 0].long()] = True
    s["cache"][~used] = float("inf")
    check(s, attend(s))


def test_a_nan_key_of_one_request_stays_there():
    s = make(4, 100, 20, 8, 4, 56)
    clean = attend(s)
    s["cache"][s["idx"][2, 3].long(), 0] = float("nan")   # key head 0
    out = attend(s)
    assert bool(out[2, :2].isnan().all())
    for r in (0, 1, 3):
        assert torch.equal(out[r], clean[r])
    assert torch.equal(out[2, 2:], clean[2, 2:])


@pytest.mark.parametrize("q_scale,scale", [(30.0, SCALE), (1e-4, SCALE), (2.0, 0.0), (2.0, -SCALE),
                                           (200.0, 0.02)])
def test_sharp_flat_zero_and_negative_scales(q_scale, scale):
    s = make(5, 900, 130, 16, 4, 60, q_scale)
    check(s, attend(s, scale=scale), scale=scale)


def test_scores_that_grow_along_the_prefix():
    """The running maximum rises all the way: every block rescales."""
    s = make(4, 2000, 64, 16, 4, 61)
    ramp = torch.linspace(0.1, 12.0, 2000, device="cuda")[:, None]
    s["prefix"][:, :4 * 128] = (s["q"][0, ::4].reshape(1, 512).float() * ramp / 8).to(torch.bfloat16)
    check(s, attend(s))
    s["prefix"][:, :4 * 128] = s["prefix"][:, :4 * 128].flip(0).contiguous()
    check(s, attend(s))


def test_long_prefix_past_32_bit_offsets():
    """A prefix of more than 2^32 bytes: its last rows are the ones that count."""
    P, h, hq = (1 << 20) + 77, 8, 8
    s = dict(R=1, P=P, k=0, hq=hq, h=h, rows=0, cache=None, idx=None)
    g = torch.Generator(device="cuda").manual_seed(3)
    s["q"] = bf16(g, 1, hq, 128)
    s["prefix"] = torch.zeros((P, h * 256), dtype=torch.bfloat16, device="cuda")
    tail = bf16(g, 50, h * 256)
    for head in range(h):                 # keys along the query: scores of about 23 against 0
        tail[:, head * 128:(head + 1) * 128] += 2 * s["q"][0, head]
    s["prefix"][-50:] = tail
    check(s, attend(s))


def test_side_stream_and_graphs_with_their_own_workspaces():
    s = make(8, 900, 100, 32, 8, 70)
    t = make(8, 900, 100, 32, 8, 71)
    want_s, want_t = attend(s), attend(t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = attend(s, stream=side)
    side.synchronize()
    assert torch.equal(got, want_s)
    need = hs.hs_prefix_attention_bytes(8, 32, 8, 900, 100)
    outs = [torch.zeros((8, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    works = [torch.zeros(max(16, need), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr, x, o, wk in zip(graphs, (s, t), outs, works):
        with torch.cuda.graph(gr):
            attend(x, out=o, work=wk)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want_s) and torch.equal(outs[1], want_t)
    s["q"].copy_(t["q"])
    graphs[0].replay()
    torch.cuda.synchronize()
    check(s, outs[0])


def test_refused_workspace_leaves_the_output_alone():
    s = make(2, 500, 10, 8, 8, 80)
    out = torch.full((2, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    need = hs.hs_prefix_attention_bytes(2, 8, 8, 500, 10)
    if need:
        with pytest.raises(hs.HsError) as e:
            hs.hs_prefix_attention(s["q"], s["prefix"], 500, s["cache"], s["rows"], s["idx"], 2, 10,
                                   8, 8, SCALE, out, out, need - 1)
        assert e.value.code == hs.HS_ERR_INVALID_ARG
    with pytest.raises(hs.HsError):
        attend(s, out=out, hq=12)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


def test_guard_bytes_around_output_and_workspace_stay():
    s = make(3, 700, 50, 24, 8, 81)
    need = hs.hs_prefix_attention_bytes(3, 24, 8, 700, 50)
    n = 3 * 24 * 128
    buf = torch.full((n + 256,), 5.0, dtype=torch.bfloat16, device="cuda")
    work = torch.full((need + 256,), 0x55, dtype=torch.uint8, device="cuda")
    hs.hs_prefix_attention(s["q"], s["prefix"], 700, s["cache"], s["rows"], s["idx"], 3, 50, 24, 8,
                           SCALE, buf[128:], work[128:], need)
    torch.cuda.synchronize()
    assert bool((buf[:128] == 5.0).all()) and bool((buf[128 + n:] == 5.0).all())
    assert bool((work[:128] == 0x55).all()) and bool((work[128 + need:] == 0x55).all())
    check(s, buf[128:128 + n].view(3, 24, 128))

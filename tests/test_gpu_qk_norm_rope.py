"""hs_qk_norm_rope against its definition in 64 bits (tests/token_reference.py,
where the bound is derived): head layouts, partial and interleaved rotations,
far and negative positions, strides of a fused projection, scattered and
padded record rows, other streams, captured graphs, and the pool's own host
records as the destination."""
import numpy as np
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref
from workloads import configs

pytestmark = pytest.mark.gpu
EPS = 1e-6


def freqs(rot):
    return [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else []


def make(n, hq, h, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn((n, hq + 2 * h, 128), generator=g, device="cuda") * scale).to(torch.bfloat16)
    wq = (1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(torch.bfloat16)
    wk = (1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(torch.bfloat16)
    return qkv, wq, wk, g


def check(got, x, w, pos, inv_freq, interleaved, eps=EPS):
    y, size = ref.norm_rope(x, w, pos, inv_freq, eps, interleaved)
    err = (got.double() - y).abs()
    assert bool((err <= ref.norm_rope_bound(y, size)).all()), err.max().item()


def run_fused(qkv, wq, wk, pos, n, hq, h, inv_freq, inter, rows=None, pool=None, stream=None):
    """One call over a fused projection output; (q_out, records)."""
    pool = n if pool is None else pool
    q_out = torch.full((n, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    records = torch.full((pool, 2 * h, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    width = (hq + 2 * h) * 128
    d = hs.qk_desc(hq, h, inv_freq, eps=EPS, interleaved=inter, q_stride=width, k_stride=width,
                   v_stride=width)
    hs.hs_qk_norm_rope(d, qkv, qkv[:, hq:], qkv[:, hq + h:], wq, wk, pos, n, q_out, records, pool,
                       rows, stream)
    return q_out, records


@pytest.mark.parametrize("n,hq,h", [(1, 1, 1), (1, 32, 8), (3, 8, 8), (7, 10, 2), (33, 21, 7),
                                    (1000, 12, 3), (257, 128, 8)])
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, False), (32, True),
                                       (16, False), (96, False), (112, True), (0, False)])
def test_against_definition(n, hq, h, rot, inter):
    qkv, wq, wk, g = make(n, hq, h, n * 100 + hq + rot)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    q_out, records = run_fused(qkv, wq, wk, pos, n, hq, h, freqs(rot), inter)
    check(q_out, qkv[:, :hq], wq, pos, freqs(rot), inter)
    check(records[:, :h], qkv[:, hq:hq + h], wk, pos, freqs(rot), inter)
    assert torch.equal(records[:, h:].view(torch.int16), qkv[:, hq + h:].view(torch.int16))


def test_many_tokens_per_block_and_rows_scattered():
    """More units than one pass of the grid; rows in no order, some padded;
    rows that no token names stay as they were."""
    n, hq, h, pool = 20011, 16, 8, 30000
    qkv, wq, wk, g = make(n, hq, h, 5)
    pos = torch.randint(0, 1 << 17, (n,), generator=g, device="cuda", dtype=torch.int32)
    rows = torch.randperm(pool, generator=g, device="cuda")[:n]
    skip = torch.rand(n, generator=g, device="cuda") < 0.1
    rows[skip] = torch.where(torch.rand(int(skip.sum()), generator=g, device="cuda") < 0.5,
                             -1, pool).to(torch.int64)
    q_out, records = run_fused(qkv, wq, wk, pos, n, hq, h, freqs(128), False, rows, pool)
    check(q_out, qkv[:, :hq], wq, pos, freqs(128), False)
    keep = ~skip
    check(records[rows[keep], :h], qkv[keep, hq:hq + h], wk, pos[keep], freqs(128), False)
    assert torch.equal(records[rows[keep], h:], qkv[keep, hq + h:])
    untouched = torch.ones(pool, dtype=torch.bool, device="cuda")
    untouched[rows[keep]] = False
    assert bool((records[untouched] == 7.0).all())


@pytest.mark.parametrize("p", [0, 1, -1, 1048575, (1 << 31) - 1, -(1 << 31)])
def test_extreme_positions(p):
    n, hq, h = 2, 4, 2
    qkv, wq, wk, _ = make(n, hq, h, 9)
    pos = torch.full((n,), p, dtype=torch.int32, device="cuda")
    for inter in (False, True):
        q_out, records = run_fused(qkv, wq, wk, pos, n, hq, h, freqs(128), inter)
        check(q_out, qkv[:, :hq], wq, pos, freqs(128), inter)
        check(records[:, :h], qkv[:, hq:hq + h], wk, pos, freqs(128), inter)


def test_frequencies_of_any_sign_and_size():
    n, hq, h = 5, 2, 1
    qkv, wq, wk, g = make(n, hq, h, 10)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    inv = [-1.0, 7.5, 0.0, 1e-9, -1e-300, 2.0, 0.3, 100.0]
    q_out, records = run_fused(qkv, wq, wk, pos, n, hq, h, inv, False)
    check(q_out, qkv[:, :hq], wq, pos, inv, False)
    check(records[:, :h], qkv[:, hq:hq + h], wk, pos, inv, False)


def test_separate_tensors_and_no_weights_and_large_and_tiny_values():
    """Dense strides, NULL weights; heads of 1e-3 and 1e4 (whose squares' sum
    stays in fp32); a head of zeros stays zero."""
    n, hq, h = 6, 6, 3
    for scale in (1e-3, 1e4):
        qkv, _, _, g = make(n, hq, h, 12, scale)
        q, k, v = qkv[:, :hq].contiguous(), qkv[:, hq:hq + h].contiguous(), qkv[:, hq + h:].contiguous()
        q[0, 0] = 0
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        q_out = torch.empty_like(q)
        records = torch.empty((n, 2 * h, 128), dtype=torch.bfloat16, device="cuda")
        hs.hs_qk_norm_rope(hs.qk_desc(hq, h, freqs(128), eps=EPS), q, k, v, None, None, pos, n,
                           q_out, records, n)
        check(q_out, q, None, pos, freqs(128), False)
        check(records[:, :h], k, None, pos, freqs(128), False)
        assert torch.equal(records[:, h:], v)
        assert bool((q_out[0, 0] == 0).all())


def test_nan_and_infinite_heads_stay_in_their_head():
    n, hq, h = 3, 4, 2
    qkv, wq, wk, _ = make(n, hq, h, 13)
    clean = run_fused(qkv, wq, wk, torch.arange(n, dtype=torch.int32, device="cuda"), n, hq, h,
                      freqs(128), False)
    bad = qkv.clone()
    bad[1, 2, 5] = float("nan")          # a query head
    bad[2, hq, 7] = float("inf")         # a key head
    bad[0, hq + h, 3] = float("nan")     # a value: copied as it is
    q_out, records = run_fused(bad, wq, wk, torch.arange(n, dtype=torch.int32, device="cuda"), n, hq,
                               h, freqs(128), False)
    assert bool(q_out[1, 2].isnan().all())
    assert bool(records[2, 0].isnan().any())
    assert torch.equal(records[0, h].isnan(), bad[0, hq + h].isnan())
    same = torch.ones((n, hq), dtype=torch.bool, device="cuda")
    same[1, 2] = False
    assert torch.equal(q_out[same], clean[0][same])
    same = torch.ones((n, 2 * h), dtype=torch.bool, device="cuda")
    same[2, 0] = same[0, h] = False
    assert torch.equal(records[same], clean[1][same])


def test_side_stream_and_captured_graph():
    n, hq, h = 64, 16, 4
    qkv, wq, wk, g = make(n, hq, h, 14)
    pos = torch.randint(0, 1 << 18, (n,), generator=g, device="cuda", dtype=torch.int32)
    want = run_fused(qkv, wq, wk, pos, n, hq, h, freqs(128), False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run_fused(qkv, wq, wk, pos, n, hq, h, freqs(128), False, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q_out = torch.zeros((n, hq, 128), dtype=torch.bfloat16, device="cuda")
    records = torch.zeros((n, 2 * h, 128), dtype=torch.bfloat16, device="cuda")
    width = (hq + 2 * h) * 128
    d = hs.qk_desc(hq, h, freqs(128), eps=EPS, q_stride=width, k_stride=width, v_stride=width)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_qk_norm_rope(d, qkv, qkv[:, hq:], qkv[:, hq + h:], wq, wk, pos, n, q_out, records, n)
    del d                                # the descriptor is read by the call, not kept
    new, _, _, _ = make(n, hq, h, 15)
    qkv.copy_(new)
    pos += 3
    graph.replay()
    torch.cuda.synchronize()
    check(q_out, new[:, :hq], wq, pos, freqs(128), False)
    check(records[:, :h], new[:, hq:hq + h], wk, pos, freqs(128), False)


def test_refusals_leave_the_outputs_alone():
    n, hq, h = 4, 4, 2
    qkv, wq, wk, _ = make(n, hq, h, 16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q_out = torch.full((n, hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    records = torch.full((n, 2 * h, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    d = hs.qk_desc(hq, h, freqs(128))
    for args in ((qkv.data_ptr() + 2, qkv, qkv), (qkv, None, qkv)):
        with pytest.raises(hs.HsError) as e:
            hs.hs_qk_norm_rope(d, *args, wq, wk, pos, n, q_out, records, n)
        assert e.value.code == hs.HS_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((q_out == 3.0).all()) and bool((records == 3.0).all())


@pytest.mark.parametrize("overlap", [hs.HS_OVERLAP_ON, hs.HS_OVERLAP_OFF])
def test_records_written_into_the_pool_reach_the_next_resolve(overlap):
    """New tokens' records written into the pool's mapped host records are what
    a resolve launched right behind, without a synchronisation, publishes."""
    R, h, hq, L = 4, 8, 16, 2000
    w = configs.QUEST_PAGES.with_(n_requests=R, n_layers=2, n_positions=L, k=64, slots=128)
    with hs.Pool.for_workload(w, launch_overlap=overlap) as pool:
        for r in range(R):
            for l in range(2):
                pool.host_records(r, l)[:] = 0
        out = torch.empty((R, w.k), dtype=torch.int32, device="cuda")
        cache = pool.views(1)["cache"]
        base = hs.hs_host_records(pool.handle, 0, 1)
        for step in range(5):
            n = R * 16                    # sixteen new tokens per request
            qkv, wq, wk, g = make(n, hq, h, 20 + step)
            at = 300 * step + 100 + torch.arange(16, device="cuda")
            pos = at.repeat(R).to(torch.int32)
            rows = (torch.arange(R, device="cuda").repeat_interleave(16) * L + pos).to(torch.int64)
            q_out = torch.empty((n, hq, 128), dtype=torch.bfloat16, device="cuda")
            width = (hq + 2 * h) * 128
            d = hs.qk_desc(hq, h, freqs(128), eps=EPS, q_stride=width, k_stride=width, v_stride=width)
            sel = (300 * step + 80 + torch.arange(w.k, device="cuda")).repeat(R, 1).to(torch.int32)
            torch.cuda.synchronize()
            hs.hs_qk_norm_rope(d, qkv, qkv[:, hq:], qkv[:, hq + h:], wq, wk, pos, n, q_out, base,
                               R * L, rows)
            pool.resolve(1, sel, out)
            torch.cuda.synchronize()
            got = cache[out[:, 20:36].long()].view(torch.bfloat16).view(n, 2 * h, 128)
            check(got[:, :h], qkv[:, hq:hq + h], wk, pos, freqs(128), False)
            assert torch.equal(got[:, h:], qkv[:, hq + h:])
        assert pool.stats()["status"] == 0
        assert np.all(pool.host_records(0, 0) == 0)

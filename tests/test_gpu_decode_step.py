"""The decode-step operators together, as a serving loop uses them: a new
token's queries and record (hs_qk_norm_rope, into the pool's host records),
the resolve of the selection, attention over a shared prefix and the published
rows and attention with accumulated weights, and the next selection from them
(hs_select_heavy) -- all enqueued on one stream with no synchronisation in
between -- against the definitions in 64 bits fed with the GPU's own
selections."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref
from workloads import configs, records

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
FREQ = [10000.0 ** (-i / 64) for i in range(64)]


@pytest.mark.parametrize("R,h,group,k,recent", [(3, 8, 1, 64, 8), (4, 8, 4, 160, 16)])
def test_decode_steps(R, h, group, k, recent):
    hq, L, start, steps, P = h * group, 1200, 700, 6, 333
    w = configs.QUEST_PAGES.with_(n_requests=R, n_layers=1, n_positions=L, k=k, slots=2 * k,
                                  record_bytes=h * 512)
    g = torch.Generator(device="cuda").manual_seed(R)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    qkv = bf16(steps, R, hq + 2 * h, 128)
    wq, wk = bf16(128), bf16(128)
    prefix = bf16(P, h * 256)
    weights = torch.zeros((R, L), device="cuda")
    sels = torch.zeros((steps + 1, R, k), dtype=torch.int32, device="cuda")
    sels[0] = torch.arange(start + 1 - k, start + 1, device="cuda", dtype=torch.int32)
    rows = torch.empty((steps, R, k), dtype=torch.int32, device="cuda")
    q = torch.empty((steps, R, hq, 128), dtype=torch.bfloat16, device="cuda")
    o_prefix, o_own = torch.empty_like(q), torch.empty_like(q)
    acc = torch.empty((steps, R, L), device="cuda")
    pos = torch.arange(start, start + steps, device="cuda", dtype=torch.int32)[:, None].repeat(1, R)
    at = (torch.arange(R, device="cuda") * L + pos).to(torch.int64)
    width = (hq + 2 * h) * 128
    desc = hs.qk_desc(hq, h, FREQ, q_stride=width, k_stride=width, v_stride=width)
    b1 = hs.hs_prefix_attention_bytes(R, hq, h, P, k)
    b2 = hs.hs_attention_weights_bytes(R, hq, h, k)
    w1 = torch.empty(max(16, b1), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(max(16, b2), dtype=torch.uint8, device="cuda")
    with hs.Pool.for_workload(w) as pool:
        for r in range(R):
            records.fill(pool.host_records(r, 0).ctypes.data, w, r, 0)
        host = hs.hs_host_records(pool.handle, 0, 0)
        cache = pool.views(0)["cache"]
        torch.cuda.synchronize()
        for t in range(steps):
            x = qkv[t]
            hs.hs_qk_norm_rope(desc, x, x[:, hq:], x[:, hq + h:], wq, wk, pos[t], R, q[t], host,
                               R * L, at[t])
            pool.resolve(0, sels[t], rows[t])
            hs.hs_prefix_attention(q[t], prefix, P, cache, cache.shape[0], rows[t], R, k, hq, h,
                                   SCALE, o_prefix[t], w1, b1)
            hs.hs_sparse_attention_weights(q[t], cache, cache.shape[0], rows[t], sels[t], R, k, hq,
                                           h, SCALE, o_own[t], weights, R, L, w2, b2)
            acc[t].copy_(weights)
            # positions 0 .. start + t exist; the next step adds one more
            hs.hs_select_heavy(weights, R, L, pos[t] + 2, R, k, recent, sels[t + 1])
        torch.cuda.synchronize()
        assert pool.stats()["status"] == 0
        all_rec = torch.stack([torch.from_numpy(pool.host_records(r, 0).copy()) for r in range(R)])
    all_rec = all_rec.cuda().view(torch.bfloat16).view(R, L, h * 256)
    total = torch.zeros((R, L), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(total)
    for t in range(steps):
        y, size = ref.norm_rope(qkv[t, :, :hq], wq, pos[t], FREQ, 1e-6, False)
        assert bool(((q[t].double() - y).abs() <= ref.norm_rope_bound(y, size)).all())
        new = all_rec[torch.arange(R), start + t].view(R, 2 * h, 128)
        y, size = ref.norm_rope(qkv[t, :, hq:hq + h], wk, pos[t], FREQ, 1e-6, False)
        assert bool(((new[:, :h].double() - y).abs() <= ref.norm_rope_bound(y, size)).all())
        assert torch.equal(new[:, h:], qkv[t, :, hq + h:])
        for r in range(R):
            sel = sels[t, r].long()
            assert sel.unique().numel() == k and int(sel.max()) == start + t
            keys, values = ref.split(all_rec[r, sel], h)
            want, p, bound, rel = ref.attention(q[t, r], keys, values, SCALE)
            assert bool(((o_own[t, r].double() - want).abs() <= bound).all()), (t, r)
            total[r, sel] += p.sum(0)
            tol[r, sel] += p.sum(0) * (rel + 2.0 ** -17)
            keys, values = ref.split(torch.cat((prefix, all_rec[r, sel])), h)
            want, _, bound, _ = ref.attention(q[t, r], keys, values, SCALE)
            assert bool(((o_prefix[t, r].double() - want).abs() <= bound).all()), (t, r)
            assert bool(((acc[t, r].double() - total[r]).abs() <= tol[r] + 2.0 ** -23 * steps * total[r]).all())
            kept = ref.keep(acc[t, r].tolist(), start + t + 2, k, recent)
            assert sels[t + 1, r].tolist() == kept, (t, r)

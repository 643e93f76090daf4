"""hs_sparse_attention_weights where a request's softmax is not a number: its
valid rows' positions and its outputs become NaN, masked rows still add
nothing, and the other requests stay as they are."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["query", "key"])
@pytest.mark.parametrize("R,k,hq,h", [(3, 90, 8, 8), (3, 700, 24, 4), (40, 2048, 32, 8)])
def test_masked_rows_add_nothing_beside_nan(R, k, hq, h, where, bad):
    g = torch.Generator(device="cuda").manual_seed(k)
    q = torch.randn((R, hq, 128), generator=g, device="cuda").to(torch.bfloat16)
    rows, L = R * k, 4000
    cache = torch.randn((rows, h * 256), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.randperm(rows, generator=g, device="cuda").view(R, k).to(torch.int32)
    sel = torch.stack([torch.randperm(L, generator=g, device="cuda")[:k] for _ in range(R)])
    sel = sel.to(torch.int32).contiguous()
    idx[:, 1::3] = -1
    idx[:, 2::9] = rows
    before = torch.rand((R, L), generator=g, device="cuda")
    need = hs.hs_attention_weights_bytes(R, hq, h, k)

    def run():
        acc = before.clone()
        out = torch.empty((R, hq, 128), dtype=torch.bfloat16, device="cuda")
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        hs.hs_sparse_attention_weights(q, cache, rows, idx, sel, R, k, hq, h, 128 ** -0.5, out, acc,
                                       R, L, work, need)
        return out, acc

    clean_out, clean = run()
    head = hq // h - 1                   # of key-value head 0
    if where == "query":
        q[1, head] = bad                 # inf: products of both signs, whose sum is NaN
    else:
        # inf: a score of infinity (of either sign, by query); the softmax of a
        # query that meets +inf is not a number
        cache[idx[1, 0].long(), 0] = bad
        q[1, head, 0] = 1.0
    out, acc = run()
    assert bool(out[1, head].isnan().all())
    valid = (idx[1] >= 0) & (idx[1] < rows)
    masked = sel[1][~valid].long()
    assert torch.equal(acc[1, masked], before[1, masked])
    assert bool(acc[1, sel[1, 0].long()].isnan())
    other = [r for r in range(R) if r != 1]
    assert torch.equal(acc[other], clean[other]) and torch.equal(out[other], clean_out[other])

"""hs_sparse_attention_weights against its definition in 64 bits
(tests/token_reference.py, where the bounds are derived): the output and the
running sums of every position's attention weight, at selection sizes around
the tile sizes, head layouts, masked rows, request ids, positions that are out
of range, repeated calls and captured graphs."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import token_reference as ref

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def make(R, k, hq, h, seed, positions=3001, q_scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def bf16(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    rows = R * k + 5
    positions = max(positions, k)
    return dict(R=R, k=k, hq=hq, h=h, L=positions, q=bf16(R, hq, 128, scale=q_scale), rows=rows,
                cache=bf16(rows, h * 256),
                idx=torch.randperm(rows, generator=g, device="cuda")[:R * k].view(R, k)
                .to(torch.int32).contiguous(),
                sel=torch.stack([torch.randperm(positions, generator=g, device="cuda")[:k]
                                 for _ in range(R)]).to(torch.int32),
                acc=torch.rand((R, positions), generator=g, device="cuda"))


def attend(s, acc, out=None, work=None, req_ids=None, weight_rows=None, stream=None):
    if out is None:
        out = torch.full((s["R"], s["hq"], 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    need = hs.hs_attention_weights_bytes(s["R"], s["hq"], s["h"], s["k"])
    if work is None:
        work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    hs.hs_sparse_attention_weights(s["q"], s["cache"], s["rows"], s["idx"], s["sel"], s["R"], s["k"],
                                   s["hq"], s["h"], SCALE, out, acc,
                                   acc.shape[0] if weight_rows is None else weight_rows, s["L"],
                                   work, need, req_ids, stream)
    return out


def check(s, out, acc, before, req_ids=None):
    want = before.double()
    tol = torch.zeros_like(want)
    for r in range(s["R"]):
        idx = s["idx"][r].long()
        ok = (idx >= 0) & (idx < s["rows"])
        keys, values = ref.split(s["cache"][idx[ok]], s["h"])
        o, p, bound, rel = ref.attention(s["q"][r], keys, values, SCALE)
        err = (out[r].double() - o).abs()
        assert bool((err <= bound).all()), (r, (err - bound).max().item())
        req = r if req_ids is None else req_ids[r]
        pos = s["sel"][r].long()[ok]
        if not 0 <= req < acc.shape[0]:
            continue
        inside = (pos >= 0) & (pos < s["L"])
        w = p.sum(0)[inside]
        want[req].index_add_(0, pos[inside], w)
        # the head sum has fewer than 128 additions; then one more per addition
        # to the running sum (counted once per call here)
        tol[req].index_add_(0, pos[inside], w * (rel + 128 * 2.0 ** -24))
    tol += 2.0 ** -23 * want.abs()
    # below the smallest normal fp32 number, 2^-126, the relative bounds end:
    # an exponential, a product or an addition (a global atomic one flushes)
    # may lose up to 2^-126, and there are at most three per query head and one
    # per addition to the running sum
    tiny = (3 * s["hq"] + s["R"]) * 2.0 ** -126
    tol += torch.where(tol > 2.0 ** -23 * want.abs(), tiny, 0.0)
    err = (acc.double() - want).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()
    touched = torch.zeros_like(want, dtype=torch.bool)
    for r in range(s["R"]):
        req = r if req_ids is None else req_ids[r]
        if 0 <= req < acc.shape[0]:
            pos = s["sel"][r].long()
            touched[req, pos[(pos >= 0) & (pos < s["L"])]] = True
    assert torch.equal(acc[~touched], before[~touched])


@pytest.mark.parametrize("R,k,hq,h", [
    (1, 1, 1, 1), (1, 64, 8, 8), (3, 33, 8, 8), (2, 65, 16, 4), (5, 777, 6, 2), (7, 16, 15, 5),
    (4, 1000, 64, 8), (40, 96, 4, 2), (1, 2048, 32, 8), (33, 300, 128, 8), (160, 40, 8, 4),
    (2, 4097, 48, 3), (1, 30000, 128, 8), (32, 2048, 32, 8)])
def test_against_definition(R, k, hq, h):
    s = make(R, k, hq, h, R * 100 + k)
    acc = s["acc"].clone()
    out = attend(s, acc)
    check(s, out, acc, s["acc"])
    acc2 = s["acc"].clone()
    out2 = attend(s, acc2)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert torch.equal(acc.view(torch.int32), acc2.view(torch.int32))


@pytest.mark.parametrize("h", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", [1, 3, 4, 8, 9, 16])
def test_head_layouts(h, group):
    s = make(3, 150, h * group, h, h * 100 + group)
    acc = s["acc"].clone()
    check(s, attend(s, acc), acc, s["acc"])


def test_masked_rows_add_nothing():
    s = make(5, 200, 16, 8, 4)
    s["idx"][0] = -1
    s["idx"][1, ::3] = s["rows"]
    s["idx"][2, 1:] = -1
    s["idx"][3, :64] = -7
    acc = s["acc"].clone()
    out = attend(s, acc)
    assert bool((out[0] == 0).all())
    assert torch.equal(acc[0], s["acc"][0])
    check(s, out, acc, s["acc"])


def test_request_ids_and_positions_out_of_range():
    s = make(4, 90, 16, 4, 5)
    ids = [7, -1, 2, 9]
    before = torch.rand((9, s["L"]), device="cuda")
    s["sel"][0, 5] = -1
    s["sel"][2, 6] = s["L"]
    s["sel"][2, 7] = 1 << 30
    acc = before.clone()
    out = attend(s, acc, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
    check(s, out, acc, before, ids)


def test_a_repeated_position_and_a_shared_request_receive_every_addition():
    s = make(3, 40, 8, 4, 6)
    s["sel"][1, 10:20] = s["sel"][1, 10]
    acc = s["acc"].clone()
    out = attend(s, acc)
    check(s, out, acc, s["acc"])
    ids = [1, 1, 1]
    acc = s["acc"].clone()
    out = attend(s, acc, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
    check(s, out, acc, s["acc"], ids)


def test_sums_run_on_over_calls_and_total_to_the_heads():
    """Each call adds a total of one per query head and request."""
    s = make(4, 300, 32, 8, 7)
    acc = torch.zeros((4, s["L"]), device="cuda")
    for step in range(1, 6):
        attend(s, acc)
        # 300 weights, each within its bound of about 2^-10, sum to 32 a call
        assert torch.allclose(acc.double().sum(1), torch.full((4,), 32.0 * step, dtype=torch.float64,
                                                              device="cuda"), rtol=1e-3)


def test_sharp_scores():
    s = make(3, 500, 16, 4, 8, q_scale=40.0)
    acc = torch.zeros_like(s["acc"])
    check(s, attend(s, acc), acc, torch.zeros_like(acc))


def test_captured_graphs_with_their_own_workspaces():
    s, t = make(8, 600, 32, 8, 9), make(8, 600, 32, 8, 10)
    accs = [torch.zeros_like(s["acc"]), torch.zeros_like(t["acc"])]
    wants = []
    for x in (s, t):
        a = torch.zeros_like(x["acc"])
        wants.append((attend(x, a), a))
    need = hs.hs_attention_weights_bytes(8, 32, 8, 600)
    outs = [torch.zeros((8, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    works = [torch.zeros(max(16, need), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr, x, a, o, wk in zip(graphs, (s, t), accs, outs, works):
        with torch.cuda.graph(gr):
            attend(x, a, out=o, work=wk)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for gr, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            gr.replay()
    torch.cuda.synchronize()
    for (o, a), got, acc in zip(wants, outs, accs):
        assert torch.equal(o, got) and torch.equal(a, acc)


def test_refusal_leaves_everything_alone():
    s = make(2, 50, 8, 8, 11)
    acc = s["acc"].clone()
    out = torch.full((2, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hs.HsError) as e:
        hs.hs_sparse_attention_weights(s["q"], s["cache"], s["rows"], s["idx"], s["sel"], 2, 50, 12, 8,
                                       SCALE, out, acc, 2, s["L"], out, 1 << 30)
    assert e.value.code == hs.HS_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(acc, s["acc"]) and bool((out == 3.0).all())

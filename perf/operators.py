"""What the operators of a decode step over per-head token records cost.

A token record holds the bf16 keys of ``heads`` key-value heads of 128
dimensions, then their values: heads * 512 bytes.  Four operators:

``qk``       per-head RMS norm of queries and keys with the position rotation,
             writing the queries and the token's record;
``prefix``   attention of a batch over a prefix that all its requests share
             and over each request's own published rows;
``weights``  attention over the published rows that also adds every row's
             attention weight to its position's running sum;
``select``   the positions a request keeps: its most recent ones and those of
             the largest accumulated weight.
"""
import math

import torch

own = False  # the tools set it: false computes the plain forms, true calls the framework

D = 128


def listed():
    return [
        # one decode step of 8 requests: each new token's record goes to its place in a pool
        {"name": "qk_decode_8", "op": "qk", "tokens": 8, "q_heads": 32, "heads": 8, "rot": 128,
         "interleaved": False, "pool": 4096, "pad": 0, "pos0": 131000},
        # an odd prefill chunk far into a long context, half-rotated heads, padding tokens at the end
        {"name": "qk_chunk_1021", "op": "qk", "tokens": 1021, "q_heads": 10, "heads": 2, "rot": 64,
         "interleaved": True, "pool": 1500, "pad": 13, "pos0": 1040000},
        # a long prefill: one 32768-token context, 32 query and 8 key-value heads
        {"name": "qk_prefill_32768", "op": "qk", "tokens": 32768, "q_heads": 32, "heads": 8, "rot": 128,
         "interleaved": False, "pool": 32768, "pad": 0, "pos0": 0},
        # two requests behind a short system prompt: latency counts
        {"name": "prefix_2x517", "op": "prefix", "requests": 2, "prefix": 517, "k": 33, "q_heads": 8,
         "heads": 8, "masked": 0.0},
        # nothing but the shared document, three query heads to a key-value head, odd sizes
        {"name": "prefix_19x20011", "op": "prefix", "requests": 19, "prefix": 20011, "k": 0, "q_heads": 12,
         "heads": 4, "masked": 0.0},
        # 32 questions on one 32768-token document, each with its own 512 selected rows
        {"name": "prefix_32x32768", "op": "prefix", "requests": 32, "prefix": 32768, "k": 512, "q_heads": 32,
         "heads": 8, "masked": 0.0},
        # a full batch on a 128K-token prefix with a full selection each, some rows rejected
        {"name": "prefix_64x131072", "op": "prefix", "requests": 64, "prefix": 131072, "k": 2048,
         "q_heads": 64, "heads": 8, "masked": 0.02},
        # one request, one small selection: latency counts
        {"name": "weights_1x64", "op": "weights", "requests": 1, "positions": 4096, "k": 64, "q_heads": 8,
         "heads": 8, "masked": 0.0},
        # odd selections with rejected rows, three query heads to a key-value head
        {"name": "weights_5x777", "op": "weights", "requests": 5, "positions": 20000, "k": 777, "q_heads": 6,
         "heads": 2, "masked": 0.1},
        # 32 requests with the page-wise selection's 2048 rows each
        {"name": "weights_32x2048", "op": "weights", "requests": 32, "positions": 32768, "k": 2048,
         "q_heads": 32, "heads": 8, "masked": 0.0},
        # 32 requests of a 32K context keep 2048 positions
        {"name": "select_32x32768", "op": "select", "requests": 32, "positions": 32768, "k": 2048,
         "recent": 64, "ragged": True},
        # 8 requests of a million positions
        {"name": "select_8x1048576", "op": "select", "requests": 8, "positions": 1048576, "k": 2048,
         "recent": 64, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "prefix", "weights", "select"])
    heads = rng.randint(1, 8)
    group = rng.randint(1, 8)
    if op == "qk":
        tokens = _log(rng, 1, 16384)
        pad = rng.choice([0, 0, rng.randint(0, tokens // 8)])
        return {"op": op, "tokens": tokens, "q_heads": heads * min(group, 4), "heads": heads,
                "rot": rng.choice([128, 128, 64, 32, 96]), "interleaved": rng.random() < 0.3,
                "pool": tokens + rng.randint(0, 4096), "pad": pad, "pos0": _log(rng, 1, 1 << 20) - 1}
    if op == "prefix":
        requests = _log(rng, 1, 64)
        return {"op": op, "requests": requests, "prefix": _log(rng, 1, 65536),
                "k": rng.choice([0, _log(rng, 1, 2048)]), "q_heads": heads * group, "heads": heads,
                "masked": rng.choice([0.0, 0.0, 0.05])}
    if op == "weights":
        return {"op": op, "requests": _log(rng, 1, 32), "positions": _log(rng, 4096, 131072),
                "k": _log(rng, 1, 2048), "q_heads": heads * min(group, 4), "heads": heads,
                "masked": rng.choice([0.0, 0.0, 0.05])}
    positions = _log(rng, 256, 1 << 20)
    k = min(_log(rng, 16, 4096), positions)
    return {"op": op, "requests": min(_log(rng, 1, 64), max(1, (1 << 23) // positions)),
            "positions": positions, "k": k, "recent": rng.randint(0, min(k, 256)),
            "ragged": rng.random() < 0.5}


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _rows(n_req, k, masked, g):
    """The published rows of n_req requests (each its own range of a cache of
    n_req * slots rows, in no order) and the cache's row count."""
    slots = max(1, 2 * k)
    idx = torch.rand((n_req, slots), generator=g, device="cuda").argsort(1)[:, :k]
    idx = (idx + torch.arange(n_req, device="cuda")[:, None] * slots).to(torch.int32)
    if masked and k:
        idx[torch.rand((n_req, k), generator=g, device="cuda") < masked] = -1
    return idx.contiguous(), n_req * slots


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "qk":
        n, hq, h, rot = case["tokens"], case["q_heads"], case["heads"], case["rot"]
        s["qkv"] = _normal((n, (hq + 2 * h) * D), g)          # the fused projection's output
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        s["eps"] = 1e-6
        s["inv_freq"] = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
        jitter = torch.randint(0, 3, (n,), generator=g, device="cuda")
        s["pos"] = (case["pos0"] + torch.arange(n, device="cuda") * 2 + jitter).to(torch.int32)
        rows = torch.rand(case["pool"], generator=g, device="cuda").argsort()[:n]
        if case["pad"]:
            rows[n - case["pad"]:] = -1                        # padding tokens have no record
        s["rows"] = rows.contiguous()
        s["records"] = _normal((case["pool"], 2 * h * D), g)
        s["q_out"] = torch.zeros((n, hq, D), dtype=torch.bfloat16, device="cuda")
        if own:
            from hierarchical_kv_cache_resolve_gb300 import hs
            width = (hq + 2 * h) * D
            s["desc"] = hs.qk_desc(hq, h, s["inv_freq"], eps=s["eps"], interleaved=case["interleaved"],
                                   q_stride=width, k_stride=width, v_stride=width)
        return s
    if op == "select":
        n, length, k = case["requests"], case["positions"], case["k"]
        # accumulated softmax weights: heavy-tailed, and exactly 0 where nothing was ever selected
        w = torch.exp(2.5 * torch.randn((n, length), generator=g, device="cuda") - 6)
        w[torch.rand((n, length), generator=g, device="cuda") < 0.4] = 0
        s["weights"] = w
        least = max(1, length // 2) if case["ragged"] else length
        s["lens"] = torch.randint(least, length + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["sel"] = torch.zeros((n, k), dtype=torch.int32, device="cuda")
        return s
    n, hq, h, k = case["requests"], case["q_heads"], case["heads"], case["k"]
    s["q"] = _normal((n, hq, D), g, 2.0)
    s["scale"] = D ** -0.5
    s["idx"], s["cache_rows"] = _rows(n, k, case["masked"], g)
    s["cache"] = _normal((s["cache_rows"], 2 * h * D), g)
    s["out"] = torch.zeros((n, hq, D), dtype=torch.bfloat16, device="cuda")
    if op == "prefix":
        s["prefix_rows"] = _normal((case["prefix"], 2 * h * D), g)
        if own:
            from hierarchical_kv_cache_resolve_gb300 import hs
            s["bytes"] = hs.hs_prefix_attention_bytes(n, hq, h, case["prefix"], k)
            s["work"] = torch.empty(max(16, s["bytes"]), dtype=torch.uint8, device="cuda")
    else:
        length = case["positions"]
        s["sel"] = torch.rand((n, length), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
        s["acc"] = torch.rand((n, length), generator=g, device="cuda") * 0.1
        if own:
            from hierarchical_kv_cache_resolve_gb300 import hs
            s["bytes"] = hs.hs_attention_weights_bytes(n, hq, h, k)
            s["work"] = torch.empty(max(16, s["bytes"]), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    if own:
        return _own(s)
    return {"qk": _plain_qk, "prefix": _plain_prefix, "weights": _plain_weights,
            "select": _plain_select}[s["op"]](s)


def _own(s):
    from hierarchical_kv_cache_resolve_gb300 import hs
    op = s["op"]
    if op == "qk":
        qkv, hq, h = s["qkv"], s["q_heads"], s["heads"]
        hs.hs_qk_norm_rope(s["desc"], qkv, qkv[:, hq * D:], qkv[:, (hq + h) * D:], s["wq"], s["wk"],
                           s["pos"], s["tokens"], s["q_out"], s["records"], s["pool"], s["rows"])
        return {"q": s["q_out"], "records": s["records"]}
    if op == "prefix":
        hs.hs_prefix_attention(s["q"], s["prefix_rows"], s["prefix"], s["cache"], s["cache_rows"], s["idx"],
                               s["requests"], s["k"], s["q_heads"], s["heads"], s["scale"], s["out"],
                               s["work"], s["bytes"])
        return s["out"]
    if op == "weights":
        hs.hs_sparse_attention_weights(s["q"], s["cache"], s["cache_rows"], s["idx"], s["sel"], s["requests"],
                                       s["k"], s["q_heads"], s["heads"], s["scale"], s["out"], s["acc"],
                                       s["requests"], s["positions"], s["work"], s["bytes"])
        return {"out": s["out"], "acc": s["acc"]}
    hs.hs_select_heavy(s["weights"], s["requests"], s["positions"], s["lens"], s["requests"], s["k"],
                       s["recent"], s["sel"])
    return s["sel"]


# ---- plain forms -----------------------------------------------------------

def _rotate(x, cos, sin, rot, interleaved):
    """Pairs of the first `rot` dimensions of x [n][heads][128] turned by the
    angles whose cosines and sines are [n][1][rot / 2]."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_qk(s):
    n, hq, h, rot = s["tokens"], s["q_heads"], s["heads"], s["rot"]
    x = s["qkv"].view(n, hq + 2 * h, D)
    angle = s["pos"].double()[:, None] * torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(y, w):
        y = y.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        return _rotate(y, cos, sin, rot, s["interleaved"]).to(torch.bfloat16)

    s["q_out"].copy_(one(x[:, :hq], s["wq"]))
    record = torch.cat((one(x[:, hq:hq + h], s["wk"]), x[:, hq + h:]), 1).view(n, 2 * h * D)
    keep = n - s["pad"]
    s["records"][s["rows"][:keep]] = record[:keep]
    return {"q": s["q_out"], "records": s["records"]}


def _own_rows(s):
    """Scores [n][heads][group][k] (-inf where a row is masked) and values
    [n][heads][k][128] of the requests' published rows."""
    n, hq, h, k = s["requests"], s["q_heads"], s["heads"], s["k"]
    use = (s["idx"] >= 0) & (s["idx"] < s["cache_rows"])
    rec = s["cache"][s["idx"].long().clamp(0, s["cache_rows"] - 1)].float().view(n, k, 2, h, D)
    q = s["q"].float().view(n, h, hq // h, D)
    keys, values = rec[:, :, 0].permute(0, 2, 3, 1), rec[:, :, 1].permute(0, 2, 1, 3)
    scores = torch.matmul(q, keys) * s["scale"]
    return scores.masked_fill(~use[:, None, None], float("-inf")), values


def _plain_prefix(s):
    n, hq, h, p = s["requests"], s["q_heads"], s["heads"], s["prefix"]
    rec = s["prefix_rows"].float().view(p, 2, h, D)
    q = s["q"].float().view(n, h, hq // h, D)
    rows = q.permute(1, 0, 2, 3).reshape(h, -1, D)
    shared = torch.matmul(rows, rec[:, 0].permute(1, 2, 0)) * s["scale"]      # [h][n * group][p]
    most = shared.max(-1, keepdim=True).values
    if s["k"]:
        scores, values = _own_rows(s)
        scores = scores.permute(1, 0, 2, 3).reshape(h, -1, s["k"])
        most = torch.maximum(most, scores.max(-1, keepdim=True).values)
    e = torch.exp(shared - most)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, rec[:, 1].permute(1, 0, 2))
    if s["k"]:
        e = torch.exp(scores - most)
        total = total + e.sum(-1, keepdim=True)
        mine = torch.matmul(e.view(h, n, hq // h, s["k"]).permute(1, 0, 2, 3), values)
        out = out + mine.permute(1, 0, 2, 3).reshape(h, -1, D)
    out = (out / total).view(h, n, hq // h, D).permute(1, 0, 2, 3)
    s["out"].copy_(out.reshape(n, hq, D))
    return s["out"]


def _plain_weights(s):
    n, hq = s["requests"], s["q_heads"]
    scores, values = _own_rows(s)
    most = scores.max(-1, keepdim=True).values
    e = torch.exp(scores - torch.where(most == float("-inf"), 0.0, most))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    s["out"].copy_(torch.matmul(p, values).reshape(n, hq, D))
    s["acc"].scatter_add_(1, s["sel"].long(), p.sum((1, 2)))
    return {"out": s["out"], "acc": s["acc"]}


def _plain_select(s):
    n, length, k = s["requests"], s["positions"], s["k"]
    at = torch.arange(length, device="cuda")
    lens = s["lens"].long()[:, None]
    recent = lens.clamp(max=s["recent"])
    heavy = at < lens - recent                                   # those that compete
    w = torch.where(heavy & ~torch.isnan(s["weights"]), s["weights"], float("-inf"))
    order = torch.sort(w, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at.expand(n, length))
    keep = heavy & (rank < k - recent) | (at >= lens - recent) & (at < lens)
    place = torch.where(keep, keep.cumsum(1) - 1, k)             # the kept ones in order, the rest behind
    full = torch.full((n, k + 1), -1, dtype=torch.int32, device="cuda")
    full.scatter_(1, place, at.to(torch.int32).expand(n, length))
    s["sel"].copy_(full[:, :k])
    return s["sel"]


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "qk":
        return _exact_qk(s)
    if op == "select":
        picked = []
        for r in range(case["requests"]):
            n = int(s["lens"][r])
            first = n - min(case["recent"], n)
            w = s["weights"][r, :first].double().cpu().tolist()
            heavy = sorted(range(first), key=lambda j: (-w[j], j))[:case["k"] - (n - first)]
            kept = sorted(heavy) + list(range(first, n))
            picked.append(kept + [-1] * (case["k"] - len(kept)))
        return torch.tensor(picked, dtype=torch.int32)
    n, hq, h, k = case["requests"], case["q_heads"], case["heads"], case["k"]
    g = hq // h
    out = torch.zeros((n, hq, D), dtype=torch.float64, device="cuda")
    if op == "weights":
        acc = s["acc"].double()
    for head in range(h):
        kc, vc = slice(head * D, (head + 1) * D), slice((h + head) * D, (h + head + 1) * D)
        if op == "prefix":
            pk, pv = s["prefix_rows"][:, kc].double(), s["prefix_rows"][:, vc].double()
        for r in range(n):
            ids = s["idx"][r].long()
            ok = (ids >= 0) & (ids < s["cache_rows"])
            rows = s["cache"][ids[ok]]
            keys, values = rows[:, kc].double(), rows[:, vc].double()
            if op == "prefix":
                keys, values = torch.cat((pk, keys)), torch.cat((pv, values))
            if keys.shape[0] == 0:
                continue
            q = s["q"][r, head * g:(head + 1) * g].double()
            p = torch.softmax(q @ keys.T * s["scale"], -1)
            out[r, head * g:(head + 1) * g] = p @ values
            if op == "weights":
                acc[r, s["sel"][r, ok].long()] += p.sum(0)
    return out if op == "prefix" else {"out": out, "acc": acc}


def _exact_qk(s):
    n, hq, h, rot = s["tokens"], s["q_heads"], s["heads"], s["rot"]
    x = s["qkv"].double().view(n, hq + 2 * h, D)
    heads = x[:, :hq + h]
    w = torch.cat((s["wq"].double().expand(hq, D), s["wk"].double().expand(h, D)))
    y = heads / (heads.pow(2).sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + rot // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None] * torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda"))
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    records = s["records"].double()
    for at, row in enumerate(s["rows"].tolist()):
        if row >= 0:
            records[row, :h * D] = y[at, hq:].reshape(-1)
            records[row, h * D:] = x[at, hq + h:].reshape(-1)
    return {"q": y[:, :hq].contiguous(), "records": records}


def work(case):
    op = case["op"]
    if op == "qk":
        n, hq, h = case["tokens"], case["q_heads"], case["heads"]
        read = n * (hq + 2 * h) * D * 2
        wrote = (n * hq + (n - case["pad"]) * 2 * h) * D * 2
        return {"bytes": read + wrote + n * 12, "flops": n * (hq + h) * D * 7}
    if op == "select":
        n, length, k = case["requests"], case["positions"], case["k"]
        seen = length * (3 if case["ragged"] else 4) // 4
        return {"bytes": n * (seen * 4 + k * 4 + 4), "flops": n * seen}
    n, hq, h, k = case["requests"], case["q_heads"], case["heads"], case["k"]
    rows = n * k * (1 - case["masked"])
    b = rows * h * 4 * D + n * k * 4 + n * hq * D * 2 * 2
    if op == "prefix":
        b += case["prefix"] * h * 4 * D
        return {"bytes": b, "flops": 4 * D * hq * (n * case["prefix"] + rows)}
    return {"bytes": b + n * k * 12, "flops": 4 * D * hq * rows}

"""The example of packed latent records that the package's readme gives, run as it
stands, against the definition of attention over a stretched context: the magnitude
is a temperature, every score gets its square."""
import math
import os
import re

import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
H, R, N, L, K, FACTOR = 16, 2, 150, 400, 64, 40.0


def example():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    code = max((c for c in re.findall(r"```(?:python)?\n(.*?)```", text, re.S) if "# packed latent records" in c), key=len)
    return code[code.index("# packed latent records"):]


class Checked:
    """The binding, with a look at the buffers that calls are given: their sizes
    in elements, for n queries, m records and R requests."""

    def __init__(self, x):
        self.x = x

    def __getattr__(self, name):
        return getattr(hs, name)

    def hs_unpack_records(self, packed, packed_rows, shift, records, n, rows=None, stream=None):
        assert records.numel() >= n * 576
        hs.hs_unpack_records(packed, packed_rows, shift, records, n, rows, stream)

    def hs_latent_prefill(self, *args, **kw):
        n, m, n_seq = self.x["n"], self.x["m"], self.x["n_seq"]
        need = hs.hs_latent_prefill_bytes(n, m, n_seq, H)
        out, work, size = args[11:14]
        assert out.numel() >= n * H * 128 and size >= need and (need == 0 or work.numel() >= size)
        hs.hs_latent_prefill(*args, **kw)

    def hs_packed_attention(self, *args):
        out, (work, size) = args[9], args[10:12] or (None, 0)
        assert out.numel() >= R * H * 512 and (size == 0 or work.numel() >= size)
        hs.hs_packed_attention(*args)


def run_example():
    """What the example leaves, and the queries that it was given."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def bf16(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    def every(n, step):
        return torch.arange(n + 1, dtype=torch.int32, device="cuda") * step

    n = R * N
    x = dict(torch=torch, layer=0, R=R, k=K, n=n, m=n, n_seq=R, record_rows=R * L, q=bf16(n, H, 192),
             kv=bf16(n, 576), w=bf16(512, scale=0.2) + 1, w_kv=bf16(512, H * 256, scale=512 ** -0.5),
             pos=torch.arange(N, dtype=torch.int32, device="cuda").repeat(R) + 9000, q_starts=every(R, N),
             k_starts=every(R, N), q_latent=bf16(R, H, 576))
    x["hs"] = Checked(x)
    x["rows"] = (torch.arange(R, device="cuda")[:, None] * L + torch.arange(N, device="cuda")).view(-1)
    x["places"] = x["rows"].clone()
    x["sel"] = torch.stack([torch.randperm(N, generator=g, device="cuda")[:K] for _ in range(R)]).to(torch.int32)
    x["out16"] = torch.empty_like(x["sel"])
    given = x["q"].clone()
    with hs.Pool(R, 1, L, hs.HS_PACKED_RECORD_BYTES, 2 * K, K) as pool:
        x["pool16"], x["records"] = pool, hs.hs_host_records(pool.handle, 0, 0)
        x["cache16"] = pool.views(0)["cache"]
        exec(compile(example(), "example", "exec"), x)
        torch.cuda.synchronize()
        assert pool.stats()["status"] == 0 and hs.hs_attention_status() == 0
    return x, given


def test_the_example_runs_with_buffers_that_are_large_enough():
    x, _ = run_example()
    assert bool(torch.isfinite(x["o_prompt"]).all()) and bool(torch.isfinite(x["o"]).all())


def test_the_example_agrees_with_the_definition():
    x, given = run_example()
    freq, _ = hs.hs_rope_frequencies(64, 10000.0, FACTOR, 4096)
    scale = 192 ** -0.5 * (0.1 * math.log(FACTOR) + 1) ** 2
    turned = ref.turned(given[..., 128:], x["pos"], freq, 1.0, True)[0]
    assert torch.equal(x["q"][..., :128], given[..., :128])
    assert bool(((x["q"][..., 128:].double() - turned).abs() <= ref.BF16 * turned.abs() + 2.0 ** -15).all())
    rec, wide = x["rec"], x["wide"]
    shared = ref.turned(x["kv"][:, None, 512:], x["pos"], freq, 1.0, True)[0][:, 0]
    assert bool(((rec[:, 512:].double() - shared).abs() <= ref.BF16 * shared.abs() + 2.0 ** -15).all())
    for r in range(R):
        of = slice(r * N, (r + 1) * N)
        for i in (0, 1, N // 2, N - 1):
            seen = slice(r * N, r * N + i + 1)
            for head in (0, H - 1):
                want, bound = ref.attention(x["q"][r * N + i, head][None],
                                            torch.cat((wide[seen, head, :128], rec[seen, 512:]), 1),
                                            wide[seen, head, 128:], scale, ref.BF16)
                assert bool(((x["o_prompt"][r * N + i, head].double() - want[0]).abs() <= bound[0]).all())
        keys = rec[of][x["sel"][r].long()]
        want, bound = ref.attention(x["q_latent"][r], keys, keys[:, :512], scale,
                                    torch.finfo(torch.float16).eps / 2, 2.0 ** -32)
        assert bool(((x["o"][r].double() - want).abs() <= bound).all())

"""The operators over latent token records on buffers that start on 16 bytes and no
wider boundary, and prompts whose first rows belong to no sequence: the same bits."""
import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import hs
from tests import test_gpu_latent_prefill as prefill
from tests import test_gpu_latent_records as records
from tests import test_gpu_packed_attention as packed

pytestmark = pytest.mark.gpu


def moved(x):
    """The same tensor, 16 bytes behind a wider boundary."""
    room = torch.empty(x.numel() * x.element_size() + 16, dtype=torch.uint8, device="cuda")
    y = room[16:].view(x.dtype).view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 32 == 16
    return y


def bits(x):
    return x.contiguous().view(torch.int16)


@pytest.mark.parametrize("k,h", [(1, 1), (64, 16), (300, 16), (777, 40), (500, 64), (1000, 128)])
def test_packed_attention(k, h):
    s = packed.make(3, k, h, k + h)
    s["idx"][:, ::5] = -1
    want = packed.attend(s)
    out = moved(torch.zeros_like(want))
    packed.attend(s, out=out, q=moved(s["q"]), cache=moved(s["cache"]))
    assert torch.equal(bits(out), bits(want))
    # an index on 4 bytes
    room = torch.empty(s["idx"].numel() + 1, dtype=torch.int32, device="cuda")
    room[1:] = s["idx"].view(-1)
    assert torch.equal(bits(packed.attend(s, idx=room[1:])), bits(want))


@pytest.mark.parametrize("lens,keys,h", [([150, 20], [180, 25], 3), ([300], [12000], 64), ([100], [9000], 8)])
def test_prefill(lens, keys, h):
    s = prefill.make(lens, keys, h, 4)
    want = prefill.attend(s)
    n, m, n_seq = s["n"], s["m"], len(lens)
    need = hs.hs_latent_prefill_bytes(n, m, n_seq, h)
    room = torch.zeros(need + 48, dtype=torch.uint8, device="cuda")
    assert room.data_ptr() % 32 == 0
    kv, rec, out = moved(s["kv"]), moved(s["rec"]), moved(torch.zeros_like(want))
    hs.hs_latent_prefill(moved(s["q"]), kv, kv[..., 128:], rec[:, 512:], s["qs"], s["ks"], n_seq, n, m, h,
                         prefill.SCALE, out, room[16:], need, kv_stride=h * 256, kv_head_stride=256, kr_stride=576)
    assert torch.equal(bits(out), bits(want))
    assert not bool(room[:16].any()) and not bool(room[16 + need:].any())   # nothing around the workspace


@pytest.mark.parametrize("lens,keys,h,front", [([150, 20], [180, 25], 3, 37), ([300], [12000], 64, 300),
                                               ([1, 0, 257], [9000, 3, 300], 4, 256)])
def test_rows_in_front_of_the_first_sequence(lens, keys, h, front):
    s = prefill.make([front] + lens, [50] + keys, h, 5)
    want = prefill.attend(s)
    s["qs"], s["ks"] = s["qs"][1:].clone(), s["ks"][1:].clone()
    s["lens"], s["keys"] = lens, keys
    out = torch.ones_like(want)
    s["q"][:front] = float("nan")
    s["kv"][:50] = float("nan")
    prefill.attend(s, out=out)
    assert bool((out[:front] == 1).all())
    t = prefill.make(lens, keys, h, 5)
    for name, at in (("q", front), ("kv", 50), ("rec", 50)):
        t[name] = s[name][at:].contiguous()
    # (the split goes by the sizes, so the bits of a split call may differ)
    got, apart = out[front:].double(), prefill.attend(t).double()
    assert bool(((got - apart).abs() <= 2.0 ** -6 * (1 + apart.abs())).all())
    prefill.check(t, out[front:].contiguous())


@pytest.mark.parametrize("packed_records", [False, True])
def test_norm_rope_and_packing(packed_records):
    s = records.make(77, 9, 12, True, packed=packed_records)
    t = {**s, **{name: moved(s[name]) for name in ("q", "kv", "w", "out", "records")}}
    records.call(s)
    records.call(t)
    for name in ("out", "records"):
        assert torch.equal(s[name], t[name])
    n = 77
    x = records.special_records(s["g"], n)
    a, b = torch.zeros((n, 416), dtype=torch.uint8, device="cuda"), moved(torch.zeros((n, 416), dtype=torch.uint8, device="cuda"))
    hs.hs_pack_records(x, n, 0, a, n)
    hs.hs_pack_records(moved(x), n, 0, b, n)
    assert torch.equal(a, b)
    u, v = torch.zeros_like(x), moved(torch.zeros_like(x))
    hs.hs_unpack_records(a, n, 0, u, n)
    hs.hs_unpack_records(b, n, 0, v, n)
    assert torch.equal(bits(u), bits(v))

"""CPU checks of the entry points over per-head token records: their host-side
argument checks refuse bad input before touching CUDA, the workspace sizes
are defined without a device, and the reference the GPU tests use agrees with
closed forms."""
import ctypes
import math

import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import _native, hs
from tests import token_reference as ref

INVALID = hs.HS_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return _native.load()


FREQ = [10000.0 ** (-i / 64) for i in range(64)]


def _qk(lib, desc=None, **kw):
    a = dict(q=4096, k=8192, v=12288, wq=16384, wk=20480, pos=24576, n=0, q_out=28672,
             records=32768, record_rows=10, rows=36864)
    a.update(kw)
    d = desc if desc is not None else hs.qk_desc(16, 8, FREQ)
    return lib.hs_qk_norm_rope(ctypes.byref(d), a["q"], a["k"], a["v"], a["wq"], a["wk"],
                               a["pos"], a["n"], a["q_out"], a["records"], a["record_rows"],
                               a["rows"], None)


def test_qk_norm_rope_accepts_an_empty_call(lib):
    assert _qk(lib) == hs.HS_OK
    assert _qk(lib, wq=None, wk=None, rows=None) == hs.HS_OK
    assert _qk(lib, desc=hs.qk_desc(16, 8, []), pos=None) == hs.HS_OK
    assert _qk(lib, desc=hs.qk_desc(16, 8, [-f for f in FREQ])) == hs.HS_OK
    assert _qk(lib, desc=hs.qk_desc(16, 8, FREQ, q_stride=4096, k_stride=4096, v_stride=4096)) \
        == hs.HS_OK


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(records=None), dict(pos=None),
    dict(q=4104), dict(k=8200), dict(v=12296), dict(wq=16392), dict(wk=20488), dict(pos=24578),
    dict(q_out=28680), dict(records=32776), dict(rows=36868), dict(n=-1), dict(record_rows=0),
    dict(record_rows=1 << 60)])
def test_qk_norm_rope_refuses_bad_buffers(lib, bad):
    assert _qk(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(q_heads=0), dict(q_heads=129), dict(heads=0), dict(heads=9), dict(eps=-1e-6),
    dict(eps=math.nan), dict(eps=math.inf), dict(q_stride=16 * 128 - 8), dict(k_stride=8 * 128 + 4),
    dict(v_stride=-1024), dict(q_stride=1 << 62), dict(inv_freq=FREQ[:63]),
    dict(inv_freq=[math.nan] * 64), dict(inv_freq=[math.inf] * 8)])
def test_qk_norm_rope_refuses_bad_descriptors(lib, bad):
    kw = dict(q_heads=16, heads=8, inv_freq=FREQ)
    kw.update(bad)
    assert _qk(lib, desc=hs.qk_desc(**kw)) == INVALID


def test_qk_norm_rope_refuses_a_null_descriptor_and_too_many_pairs(lib):
    assert lib.hs_qk_norm_rope(None, 16, 16, 16, None, None, 16, 0, 16, 16, 1, None, None) == INVALID
    d = hs.qk_desc(16, 8, FREQ)
    d.interleaved = 2
    assert _qk(lib, desc=d) == INVALID
    d = hs.qk_desc(16, 8, FREQ)
    d.rot_dim = 144
    assert _qk(lib, desc=d) == INVALID
    with pytest.raises(ValueError):
        hs.qk_desc(16, 8, FREQ + [1.0])


def _prefix(lib, **kw):
    a = dict(q=4096, prefix=8192, prefix_len=100, cache=12288, cache_rows=10, idx=16384, n=0, k=4,
             q_heads=16, heads=8, out=20480, work=24576, bytes=1 << 40)
    a.update(kw)
    return lib.hs_prefix_attention(a["q"], a["prefix"], a["prefix_len"], a["cache"],
                                   a["cache_rows"], a["idx"], a["n"], a["k"], a["q_heads"],
                                   a["heads"], 0.1, a["out"], a["work"], a["bytes"], None)


def test_prefix_attention_accepts_an_empty_call(lib):
    assert _prefix(lib) == hs.HS_OK
    assert _prefix(lib, k=0, cache=None, idx=None, cache_rows=0) == hs.HS_OK
    assert _prefix(lib, prefix=None, prefix_len=0) == hs.HS_OK


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(prefix=None), dict(cache=None), dict(idx=None), dict(out=None),
    dict(q=4104), dict(prefix=8200), dict(cache=12296), dict(idx=16386), dict(out=20488),
    dict(work=24584), dict(prefix_len=-1), dict(prefix_len=1 << 31), dict(cache_rows=0),
    dict(n=-1), dict(n=65536), dict(k=-1), dict(heads=0), dict(heads=9), dict(q_heads=12),
    dict(q_heads=136), dict(q_heads=17, heads=1), dict(q_heads=0)])
def test_prefix_attention_refuses(lib, bad):
    assert _prefix(lib, **bad) == INVALID


def _weights(lib, **kw):
    a = dict(q=4096, cache=12288, cache_rows=10, idx=16384, sel=28672, ids=32768, n=0, k=4,
             q_heads=16, heads=8, out=20480, acc=36864, rows=2, positions=100, work=24576,
             bytes=1 << 40)
    a.update(kw)
    return lib.hs_sparse_attention_weights(a["q"], a["cache"], a["cache_rows"], a["idx"], a["sel"],
                                           a["ids"], a["n"], a["k"], a["q_heads"], a["heads"], 0.1,
                                           a["out"], a["acc"], a["rows"], a["positions"],
                                           a["work"], a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(cache=None), dict(idx=None), dict(sel=None), dict(out=None), dict(acc=None),
    dict(q=4104), dict(cache=12296), dict(idx=16386), dict(sel=28674), dict(ids=32770),
    dict(out=20488), dict(acc=36866), dict(work=24584), dict(cache_rows=0), dict(n=-1),
    dict(n=65536), dict(k=0), dict(heads=9), dict(q_heads=12), dict(q_heads=32, heads=1),
    dict(rows=0), dict(positions=0), dict(positions=1 << 31)])
def test_sparse_attention_weights_refuses(lib, bad):
    assert _weights(lib, **bad) == INVALID


def test_sparse_attention_weights_accepts_an_empty_call(lib):
    assert _weights(lib) == hs.HS_OK
    assert _weights(lib, ids=None) == hs.HS_OK


def test_workspaces_that_are_too_small_are_refused(lib):
    need = hs.hs_attention_weights_bytes(3, 64, 8, 40000)
    assert need > 0
    assert _weights(lib, n=3, q_heads=64, k=40000, bytes=need - 1) == INVALID
    assert _weights(lib, n=3, q_heads=64, k=40000, bytes=need, work=None) == INVALID
    need = hs.hs_prefix_attention_bytes(3, 64, 8, 40000, 4)
    if need:
        assert _prefix(lib, n=3, q_heads=64, prefix_len=40000, bytes=need - 1) == INVALID
        assert _prefix(lib, n=3, q_heads=64, prefix_len=40000, bytes=need, work=None) == INVALID


def test_workspace_sizes_are_zero_for_refused_arguments():
    assert hs.hs_attention_weights_bytes(0, 8, 8, 4) == 0
    assert hs.hs_attention_weights_bytes(1, 12, 8, 4) == 0
    assert hs.hs_attention_weights_bytes(1, 8, 8, 0) == 0
    assert hs.hs_prefix_attention_bytes(1, 8, 8, 0, 0) == 0
    assert hs.hs_prefix_attention_bytes(70000, 8, 8, 10, 4) == 0
    assert hs.hs_prefix_attention_bytes(1, 8, 8, 1 << 31, 4) == 0
    assert hs.hs_prefix_attention_bytes(1, 8, 8, 100, (1 << 30) + 1) == 0


def _select(lib, **kw):
    a = dict(w=4096, rows=2, positions=100, ids=8192, lens=12288, n=0, k=10, recent=4, sel=16384)
    a.update(kw)
    return lib.hs_select_heavy(a["w"], a["rows"], a["positions"], a["ids"], a["lens"], a["n"],
                               a["k"], a["recent"], a["sel"], None)


@pytest.mark.parametrize("bad", [
    dict(w=None), dict(sel=None), dict(w=4098), dict(ids=8194), dict(lens=12290), dict(sel=16386),
    dict(rows=0), dict(positions=0), dict(positions=1 << 31), dict(n=-1), dict(n=65536), dict(k=0),
    dict(recent=-1), dict(recent=11)])
def test_select_heavy_refuses(lib, bad):
    assert _select(lib, **bad) == INVALID


def test_select_heavy_refuses_a_k_whose_loops_would_pass_31_bits(lib):
    assert _select(lib, k=1 << 30) == hs.HS_OK
    assert _select(lib, k=(1 << 30) + 1) == INVALID
    assert _select(lib, k=(1 << 31) - 1, recent=(1 << 31) - 1) == INVALID


def test_select_heavy_accepts_an_empty_call(lib):
    assert _select(lib) == hs.HS_OK
    assert _select(lib, ids=None, lens=None) == hs.HS_OK


# ---- the reference itself ---------------------------------------------------

def test_reference_norm_rope_closed_forms():
    x = torch.zeros((2, 1, 128))
    x[0, 0, 0] = 3.0                       # one element: its norm is sqrt(128) times its sign
    x[1, 0, :] = -2.0
    pos = torch.tensor([0, 5])
    y, size = ref.norm_rope(x, None, pos, [], 0.0, False)
    assert y[0, 0, 0].item() == pytest.approx(math.sqrt(128))
    assert torch.allclose(y[1], -torch.ones(1, 128, dtype=torch.float64))
    # a quarter turn maps (a, b) to (-b, a)
    pos = torch.tensor([1, 1])
    y0, _ = ref.norm_rope(x, None, pos * 0, [math.pi / 2], 0.0, False)
    y1, _ = ref.norm_rope(x, None, pos, [math.pi / 2], 0.0, False)
    assert torch.allclose(y1[..., 0], -y0[..., 1]) and torch.allclose(y1[..., 1], y0[..., 0])
    # lengths of pairs are kept
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 128), generator=g)
    for inter in (False, True):
        y, size = ref.norm_rope(x, None, torch.tensor([7, 100000, -3]), FREQ, 1e-6, inter)
        y0, _ = ref.norm_rope(x, None, torch.tensor([0, 0, 0]), FREQ, 1e-6, inter)
        a = y[..., 0::2] if inter else y[..., :64]
        b = y[..., 1::2] if inter else y[..., 64:]
        s = size[..., 0::2] if inter else size[..., :64]
        assert torch.allclose(a * a + b * b, s * s)
        assert torch.allclose((y * y).sum(-1), (y0 * y0).sum(-1))


def test_reference_attention_agrees_with_the_oracle():
    import numpy as np

    from oracle.attention import sparse_attention
    rng = np.random.default_rng(3)
    heads, n = 4, 50
    u16 = (rng.standard_normal((n, heads * 256)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    rec = torch.from_numpy(u16.view(np.int16)).view(torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((heads, 128)))
    keys, values = ref.split(rec, heads)
    out, p, bound, _ = ref.attention(q, keys, values, 0.1)
    want = sparse_attention(u16.view(np.uint8).reshape(n, -1), 1, q.numpy(), heads=heads, scale=0.1)
    assert np.allclose(out.numpy(), want, rtol=0, atol=1e-12)
    assert torch.allclose(p.sum(-1), torch.ones(heads, dtype=torch.float64))
    assert (bound > 0).all()


def test_reference_keep():
    assert ref.keep([5.0, 1.0, 5.0, 3.0, 0.0], 5, 3, 1) == [0, 2, 4]
    assert ref.keep([1.0, 1.0, 1.0, 1.0], 4, 2, 0) == [0, 1]
    assert ref.keep([math.nan, -math.inf, 2.0, 9.0], 3, 3, 0) == [0, 1, 2]
    assert ref.keep([1.0, 2.0], 2, 5, 1) == [0, 1]

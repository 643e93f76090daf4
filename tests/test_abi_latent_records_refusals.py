"""CPU checks of the entry points over latent token records at the ends of what
they accept: sizes of workspaces for refused arguments, outputs whose heads would
overlap, buffers that a call does not use."""
import ctypes

import pytest
import torch

from hierarchical_kv_cache_resolve_gb300 import _native, hs

INVALID = hs.HS_ERR_INVALID_ARG
FREQ = [10000.0 ** (-i / 32) for i in range(32)]


@pytest.fixture(scope="module")
def lib():
    return _native.load()


@pytest.mark.parametrize("n,keys", [((1 << 30) + 1, 100000), ((1 << 31) - 1, 100000), (300, (1 << 30) + 1),
                                    (300, (1 << 31) - 1)])
def test_prefill_workspace_is_zero_beyond_the_largest_sizes(n, keys):
    assert hs.hs_latent_prefill_bytes(n, keys, 1, 4) == 0
    assert hs.hs_latent_prefill_bytes(300, 1 << 30, 1, 4) > 0


def _rope(lib, desc, **kw):
    a = dict(q=4096, kv=8192, w=12288, pos=16384, n=0, q_out=20480, records=24576, rows_n=10, rows=28672)
    a.update(kw)
    return lib.hs_latent_norm_rope(ctypes.byref(desc), a["q"], a["kv"], a["w"], a["pos"], a["n"], a["q_out"],
                                   a["records"], a["rows_n"], a["rows"], None)


# the addresses are made up: the calls below have to be refused on the host
@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that was not refused would run")
@pytest.mark.parametrize("n,h,token,head", [
    (2, 2, 64, 64), (2, 2, 128, 128), (2, 3, 128, 64), (2, 2, 64, 72), (2, 2, 120, 64), (100, 16, 64 * 15, 64),
    (101, 3, 64, 6400), (7, 5, 192, 320), (1000, 128, 576, 584), (1 << 20, 2, 64, 64 << 19),
    ((1 << 31) - 1, 128, 1 << 29, 1 << 29), (4, 3, 200, 72)])
def test_outputs_that_would_overlap_are_refused(lib, n, h, token, head):
    assert _rope(lib, hs.latent_desc(h, FREQ, out_stride=token, out_head_stride=head), n=n) == INVALID


def test_overlap_is_exact():
    """The rule behind the refusals above, against every pair of pieces."""
    def overlaps(n, h, token, head):
        at = sorted(t * token + i * head for t in range(n) for i in range(h))
        return any(b - a < 64 for a, b in zip(at, at[1:]))

    def rule(n, h, token, head):
        for i in range(1, h):
            t = i * head // token
            if (t < n and i * head - t * token < 64) or (t + 1 < n and (t + 1) * token - i * head < 64):
                return True
        return False
    for n in (1, 2, 3, 7):
        for h in (1, 2, 5):
            for token in range(64, 700, 8):
                for head in (64, 72, 128, 200, 320, 576, 640):
                    assert rule(n, h, token, head) == overlaps(n, h, token, head), (n, h, token, head)


@pytest.mark.parametrize("q,q_out", [(None, None), (4100, 20484), (1, 3)])
def test_query_buffers_are_ignored_without_query_heads(lib, q, q_out):
    assert _rope(lib, hs.latent_desc(0, FREQ), q=q, q_out=q_out) == hs.HS_OK
    assert _rope(lib, hs.latent_desc(1, FREQ), q=q, q_out=q_out) == INVALID


@pytest.mark.parametrize("k", [None, 4100, 1])
def test_key_buffers_are_ignored_without_keys(lib, k):
    def call(keys):
        return lib.hs_latent_prefill(4096, k, k, k, 0, 0, 0, 20480, 24576, 2, 0, keys, 16, 0.1, 28672, 32768, 1 << 40,
                                     None)
    assert call(0) == hs.HS_OK
    assert call(1) == INVALID

"""CPU check: hs_prefix_attention ignores the cache and the indices where no
published row is asked for, whatever they are, and checks them where one is."""
import pytest

from hierarchical_kv_cache_resolve_gb300 import _native, hs


def call(k, cache, cache_rows, idx):
    return _native.load().hs_prefix_attention(4096, 8192, 100, cache, cache_rows, idx, 0, k, 16, 8, 0.1,
                                              20480, 24576, 1 << 40, None)


@pytest.mark.parametrize("cache,cache_rows,idx", [
    (12288, 10, 16384), (None, 0, None), (12296, 10, 16384), (12288, 10, 16386), (12289, -1, 16385)])
def test_cache_and_indices_are_ignored_without_rows(cache, cache_rows, idx):
    assert call(0, cache, cache_rows, idx) == hs.HS_OK
    want = hs.HS_OK if (cache, cache_rows, idx) == (12288, 10, 16384) else hs.HS_ERR_INVALID_ARG
    assert call(1, cache, cache_rows, idx) == want

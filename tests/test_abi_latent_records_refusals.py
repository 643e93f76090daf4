"""CPU checks of the entry points over latent token records at the ends of what
they accept: sizes of workspaces for refused arguments, outputs whose heads would
overlap, buffers that a call does not use."""
import ctypes

import pytest

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

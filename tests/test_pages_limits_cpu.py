"""Limits and refusals of the pages' calls that the host checks, before any launch."""
import ctypes

import pytest
import torch

from moe_speculative_decoding_gb300 import api
from moe_speculative_decoding_gb300 import build as mbuild

from test_latent_cpu import _i32, _t, entered  # noqa: F401 (a fixture: tensors of another device over no library)

UNSUPPORTED = 2


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return api.lib()


def accept(lib, seqs, heads, dtype):
    """The status of an acceptance over a cache of `heads` heads of 128 with pages of one position."""
    scales, width, pages = 4096 if dtype == 2 else None, heads * 128, 100
    kv = api.CacheDesc(4096, 4096, scales, scales, width, width, 128, dtype, heads, 128, 1, pages, 0)
    pool = api.PoolDesc(4096, 4096, 4096, pages, 1, seqs, 1)
    caches = api.CachesDesc(ctypes.addressof(kv), None, 1, 0)
    return lib.moe_pages_accept(ctypes.addressof(pool), 4096, 4096, 4096, 8, None, ctypes.addressof(caches), 4096, 1 << 60, None)


@pytest.mark.parametrize("seqs,heads,dtype", [(3 << 20, 128, 1), (1 << 20, 128, 1), ((1 << 20) + 1, 128, 1), (2 << 20, 128, 2)])
def test_accept_numbers_its_rows_in_31_bits(lib, seqs, heads, dtype):
    """Rows of 4,096 units of 16 bytes, or of 2,048 and 256 scales: 32 and 18 slices, of 64 layers each, for every
    sequence."""
    assert accept(lib, seqs, heads, dtype) == UNSUPPORTED


def test_a_cache_is_listed_once(entered):  # noqa: F811
    """Rows of one that is listed twice would move twice, those of keys that are the values too."""
    k, v, rows = _t(4, 8, 2, 4), _t(4, 8, 2, 4), _t(4, 8, 40)
    kv, latent = api.KVCache(k, v), api.LatentCache(rows, 32)
    api.page_pool([kv, latent], 2, 3)
    for caches in ([kv, kv], [latent, kv, latent], [kv, api.KVCache(k, _t(4, 8, 2, 4))], [api.KVCache(k, k)],
                   [latent, api.LatentCache(rows, 24)]):
        with pytest.raises(ValueError):
            api.page_pool(caches, 2, 3)

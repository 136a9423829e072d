"""Sizes near 2^31."""
import ctypes

import pytest
import torch

from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


def test_pages_of_nearly_2_31_positions():
    page = 2 ** 31 - 8
    z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
    refs, table, held, length = z(1), z(3, 1), z(3), z(3)
    pool = api.PoolDesc(refs.data_ptr(), table.data_ptr(), held.data_ptr(), 1, page, 3, 1)
    none = api.CachesDesc(None, None, 0, 0)
    at, caches = ctypes.addressof(pool), ctypes.addressof(none)
    ws = z(1024)
    need, count, ids = z(3), z(3), z(1) + 1
    need[0], count[0], count[1:] = page - 2, 2, -1
    s, L = torch.cuda.current_stream().cuda_stream, api.lib()
    assert L.moe_pages_reserve(at, length.data_ptr(), need.data_ptr(), None, caches, ws.data_ptr(), 4096, s) == 0
    length[0] = page - 3
    # two more positions: the last but one of the page
    assert L.moe_pages_accept(at, length.data_ptr(), None, count.data_ptr(), 2, length.data_ptr(), caches, ws.data_ptr(), 4096, s) == 0
    assert length.tolist() == [page - 1, 0, 0] and held.tolist() == [1, 0, 0] and refs.tolist() == [1]
    src = z(1)
    assert L.moe_pages_fork(at, src.data_ptr(), ids.data_ptr(), 1, length.data_ptr(), ws.data_ptr(), 4096, s) == 0
    assert length.tolist() == [page - 1, page - 1, 0] and held.tolist() == [1, 1, 0] and refs.tolist() == [2]
    assert L.moe_pages_free(at, ids.data_ptr(), 1, length.data_ptr(), ws.data_ptr(), 4096, s) == 0
    assert length.tolist() == [page - 1, 0, 0] and held.tolist() == [1, 0, 0] and refs.tolist() == [1]
    assert api.last_device_error(ws) == 0


def test_free_of_nearly_2_31_ids():
    cache = api.latent_cache(20, 4, 8, 8)
    pool = api.page_pool([cache], 2, 6)
    length = torch.tensor([9, 5], dtype=torch.int32, device="cuda")
    api.pages_reserve(pool, torch.zeros_like(length), length)
    ids = torch.full((2 ** 31 - 1,), -1, dtype=torch.int32, device="cuda")
    ids[-1] = 1
    api.pages_free(pool, ids, length)
    assert length.tolist() == [9, 0] and pool.held.tolist() == [3, 0] and int(pool.refs.sum()) == 3
    assert api.last_device_error(pool.ws) == 0

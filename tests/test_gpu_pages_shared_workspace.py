"""Forks on a workspace that other calls have used before."""
import pytest
import torch

from latent_util import LatentPass
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_forks_after_attention_on_one_workspace():
    """100 pairs take several CTAs, whose last one must not go by what an attention call left behind the header."""
    p = LatentPass([5000], [4], 16, 512, 64, 64, seed=1)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 4, 1, 16)
    pool = api.page_pool([d["cache"]], 101, 4)
    assert ws.numel() >= pool.ws_bytes
    pool.ws, pool.ws_bytes = ws, ws.numel()
    length = i32([100] + [0] * 100)
    assert api.pages_reserve(pool, i32([0] * 101), length).tolist() == [1] * 101
    for _ in range(3):
        out, lse = api.latent_attention(**d, return_lse=True, max_tokens=4, ws=ws)
        api.pages_fork(pool, i32([0] * 100), i32(list(range(1, 101))), length)
        assert api.last_device_error(ws) == 0
        assert pool.held.tolist() == [2] * 101 and length.tolist() == [100] * 101
        assert pool.refs[:2].tolist() == [101, 101] and pool.table[:, :2].tolist() == [[0, 1]] * 101
        api.pages_free(pool, i32(list(range(1, 101))), length)
    p.check(api, out, lse)

"""Latent attention of many short sequences: several items of one tile to a CTA, so that the warps which form the scores
take turns from item to item."""
import pytest
import torch

from latent_util import LatentPass
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,n", [(16, 1), (8, 4), (16, 4), (16, 3), (5, 6)])   # 16, 32 and 64 columns
@pytest.mark.parametrize("dense", [True, False])   # queries that are copied, and that threads load
def test_items_of_one_tile(heads, n, dense):
    p = LatentPass([(7 * i) % (64 - n) for i in range(900)], [n] * 900, heads, 64, 16, 8, seed=heads + n)
    d = p.device(api)
    if not dense:
        wide = torch.zeros((900 * n, heads + 1, 80), dtype=torch.bfloat16, device="cuda")
        wide[:, :heads] = d["q"]
        d["q"] = wide[:, :heads]
    ws = api.latent_attention_workspace(d["cache"], 900 * n, 900, heads)
    call = lambda: api.latent_attention(**d, return_lse=True, max_tokens=n, ws=ws)
    out, lse = call()
    assert api.last_device_error(ws) == 0
    p.check(api, out, lse)
    for _ in range(20):
        again = call()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert api.last_device_error(ws) == 0


def test_one_and_two_tiles_in_turn():
    lengths = [(1 + 61 * i) % 127 for i in range(700)]
    p = LatentPass(lengths, [1] * 700, 16, 256, 64, 16, seed=3)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 700, 700, 16)
    out, lse = api.latent_attention(**d, return_lse=True, max_tokens=1, ws=ws)
    assert api.last_device_error(ws) == 0
    p.check(api, out, lse)

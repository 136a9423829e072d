"""Lengths at the end of 31 bits: a page table may name a page many times, so that such lengths fit it.
They are refused on the device like any length that does not fit, and the batch's others keep theirs."""
import pytest
import torch

from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("cache,q_type,max_tokens", [("bf16", torch.bfloat16, 8), ("e4m3", torch.bfloat16, 8), ("bf16", torch.bfloat16, 64),
                                                     ("e4m3", torch.bfloat16, 64), ("bf16", torch.float32, 8)])
@pytest.mark.parametrize("ctx", [2 ** 31 - 1, 2 ** 31 - 60, 2 ** 31 - 127])
def test_lengths_beyond_31_bits_are_recorded(ctx, cache, q_type, max_tokens):
    page, heads, dim, n = 65536, 2, 64, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    c = api.kv_cache(1, page, 1, dim, cache)
    for i in range(0, 512, 64):
        x = torch.randn((64, 1, dim), generator=g, device=DEV)
        api.kv_write(c, x, x, torch.arange(i, i + 64, dtype=torch.int32, device=DEV))
    q = torch.randn((2 * n + 3, heads, dim), generator=g, device=DEV).to(q_type)
    table = torch.zeros((3, 32769), dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, n, 2 * n, 2 * n + 3], dtype=torch.int32, device=DEV)
    ws = api.tree_attention_workspace(c, 2 * n + 3, 3, heads)
    lengths = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 7.0), torch.full((2 * n + 3, heads), 7.0, device=DEV)
    api.tree_attention(c, q, starts, lengths(300, ctx, 400), table, max_tokens=max_tokens, out=out, lse=lse, ws=ws)
    assert api.last_device_error(ws) == 5
    assert bool((out[n:2 * n] == 7).all()) and bool((lse[n:2 * n] == 7).all())
    # the same batch with a sequence in its place that is skipped for another reason
    ref, ref_lse = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
    api.tree_attention(c, q, starts, lengths(300, -1, 400), table, max_tokens=max_tokens, out=ref, lse=ref_lse, ws=ws)
    assert api.last_device_error(ws) == 5
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert bool(out[:n].isfinite().all()) and not bool((out[:n] == 7).any()) and not bool((out[2 * n:] == 7).any())

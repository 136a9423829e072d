"""Page tables as wide as the calls take, over caches of very long pages: the bounds on a call's work go beyond 63
bits unless they are held to what a sequence can be."""
import ctypes

import pytest
import torch

from latent_util import LatentPass, within
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
PAGE, WIDE = 1 << 30, 1 << 20   # positions of a page (a tile's worth is there), page numbers of a sequence


def stream():
    return torch.cuda.current_stream().cuda_stream


def sequences(seqs, ctx):
    """One token of the first sequence, none of the others."""
    start = torch.ones(seqs + 1, dtype=torch.int32, device="cuda")
    start[0] = 0
    length = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    length[0] = ctx
    return start, length, torch.zeros((seqs, WIDE), dtype=torch.int32, device="cuda")


def test_latent_attention():
    heads, seqs = 1024, 512
    p = LatentPass([100], [1], heads, 8, 8, 128, tree=False, seed=1, spare=0)
    d = p.device(api)
    desc = api.LatentDesc.from_buffer_copy(d["cache"].desc)
    desc.page, desc.pages = PAGE, 1
    start, ctx, table = sequences(seqs, 100)
    ws = api.latent_attention_workspace(d["cache"], 1, seqs, heads)
    out, lse = torch.zeros((1, heads, 8), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, heads), device="cuda")
    code = api.lib().moe_latent_attention(ctypes.addressof(desc), api._heads(d["q"], "q", 1, heads, 16, 0), api._heads(out, "out", 1, heads, 8, 0),
                                          lse.data_ptr(), start.data_ptr(), ctx.data_ptr(), table.data_ptr(), None, seqs, 1, 64, WIDE,
                                          p.scale, ws.data_ptr(), ws.numel(), stream())
    assert code == 0 and api.last_device_error(ws) == 0
    p.check(api, out, lse)


def test_tree_attention():
    heads, seqs, n = 1024, 1024, 101
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((1, 128, heads, 8), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((1, heads, 8), generator=g).bfloat16()
    cache = api.KVCache(k.cuda(), v.cuda())
    desc = api.CacheDesc.from_buffer_copy(cache.desc)
    desc.page, desc.pages = PAGE, 1
    start, ctx, table = sequences(seqs, n - 1)
    ws = api.tree_attention_workspace(cache, 1, seqs, heads)
    dq, out = q.cuda(), torch.zeros((1, heads, 8), dtype=torch.bfloat16, device="cuda")
    code = api.lib().moe_tree_attention(ctypes.addressof(desc), api._heads(dq, "q", 1, heads, 8, 0), api._heads(out, "out", 1, heads, 8, 0), None,
                                        start.data_ptr(), ctx.data_ptr(), table.data_ptr(), None, seqs, 1, 64, WIDE, 8 ** -0.5,
                                        ws.data_ptr(), ws.numel(), stream())
    assert code == 0 and api.last_device_error(ws) == 0
    p = torch.softmax(torch.einsum("hc,phc->hp", q[0].double(), k[0, :n].double()) * 8 ** -0.5, -1)
    ref = torch.einsum("hp,phc->hc", p, v[0, :n].double())
    # the weights' rounding for the product with the values and the result's, 2^-8 each; 2^-16 for what is done in fp32
    bound = (2.0 ** -8 + 2.0 ** -16) * torch.einsum("hp,phc->hc", p, v[0, :n].double().abs())
    within("out", out[0], ref, bound + 2.0 ** -8 * (ref.abs() + bound))

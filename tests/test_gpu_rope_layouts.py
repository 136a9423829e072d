"""One rotation, whatever kernel a layout takes: the bits of fp32 rows do not depend on alignment, on
the strides, or on whether they are rotated alone, in place, or on their way into the cache."""
import pytest
import torch

from attn_util import quantise_ref
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 32), (96, 96), (256, 128)])
def test_bits_do_not_depend_on_the_layout(dim, rot, interleaved):
    g = torch.Generator(device=DEV).manual_seed(dim)
    x = torch.randn((70, 4, dim), generator=g, device=DEV)
    pos = torch.randint(500, (70,), generator=g, device=DEV).int()
    table = api.rope_table(500, *api.rope_frequencies(rot))
    for inverse in (False, True):
        base = api.rope(x, None, pos, table, interleaved=interleaved, inverse=inverse)[0]
        odd = torch.empty(x.numel() + 1, device=DEV)[1:].view(x.shape)
        odd.copy_(x)
        assert torch.equal(api.rope(odd, None, pos, table, interleaved=interleaved, inverse=inverse)[0], base)
        heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
        assert torch.equal(api.rope(None, heads_first, pos, table, interleaved=interleaved, inverse=inverse)[1], base)
        api.rope(odd, None, pos, table, interleaved=interleaved, inverse=inverse, q_out=odd)
        assert torch.equal(odd, base)
    base = api.rope(x, None, pos, table, interleaved=interleaved)[0]
    odd.copy_(x)
    slots = torch.arange(70, dtype=torch.int32, device=DEV)
    codes, scales = quantise_ref(base.cpu())
    for rows in (x, odd):
        c = api.kv_cache(9, 8, 4, dim, "f32")
        assert torch.equal(api.kv_write(c, rows, rows, slots, q=rows, positions=pos, table=table, interleaved=interleaved), base)
        assert torch.equal(c.k.view(72, 4, dim)[:70], base) and torch.equal(c.v.view(72, 4, dim)[:70], x)
        c = api.kv_cache(9, 8, 4, dim, "e4m3")
        api.kv_write(c, rows, rows, slots, positions=pos, table=table, interleaved=interleaved)
        assert torch.equal(c.k.cpu().view(72, 4, dim)[:70], codes)
        assert torch.equal(c.k_scale.cpu().transpose(1, 2).reshape(72, 4)[:70], scales)

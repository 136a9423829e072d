"""Codes of zeros and of quotients that round to zero keep their sign, as x / scale has it, whichever
kernel writes them."""
import pytest
import torch

from attn_util import quantise_ref
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [16, 64, 128, 240])
@pytest.mark.parametrize("offset", [0, 1])   # of the rows in their storage: aligned for vectors, or not
def test_negative_zeros_keep_their_sign(offset, dim, dtype):
    x = torch.randn((40, 2, dim), generator=torch.Generator().manual_seed(dim))
    x[..., 1::3] = -0.0
    x[..., 2::3] = 0.0
    x[3:6, :, 4] = -1e-7                 # rounds to zero
    x[6:9] *= 1e30                       # a scale of 2^91
    x[6:9, :, 4] = -1e-20                # whose quotient underflows
    x[9] = -0.0                          # a row of zeros
    x = x.to(dtype)
    flat = torch.empty(x.numel() + offset, dtype=dtype, device=DEV)
    rows = flat[offset:].view(x.shape)
    rows.copy_(x)
    c = api.kv_cache(5, 8, 2, dim, "e4m3")
    api.kv_write(c, rows, rows, torch.arange(40, dtype=torch.int32, device=DEV))
    codes, scales = quantise_ref(x.float())
    assert bool((codes == 0x80).any()) and bool((codes == 0).any())
    for got, got_scales in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert torch.equal(got.cpu().view(codes.shape), codes)
        assert torch.equal(got_scales.cpu().transpose(1, 2).reshape(scales.shape), scales)

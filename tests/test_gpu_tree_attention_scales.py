"""Tree attention over e4m3 codes where value scales lie far apart: a drafted token's scale must not be
felt by the rows that do not see it, nor a context position's by rows that give it no weight.  On the
kernel for few rows (the bound on the tokens is exact) and on the one for many."""
import numpy as np
import pytest
import torch

from attn_util import Pass, assert_within, quantise_ref, weight_eps
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


def _check(p, few):
    out, lse = api.tree_attention(**p.device(api), max_tokens=max(p.n) if few else 64, return_lse=True)
    ref, ref_lse, ob, lb = p.reference(weight_eps(p), True)
    assert_within("lse", lse, ref_lse, lb)
    assert_within("out", out, ref, ob)


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [3, 7, 15])   # 12, 28 and 60 rows of a key head
@pytest.mark.parametrize("huge", [17, 25, 60, 100])
def test_scale_of_a_draft_that_others_do_not_see(huge, n, dim, few):
    """A drafted token with a value scale of 2^huge that only the token itself sees."""
    p = Pass([4000, 30, 0], [n, 2, n], 8, 2, dim, 16, "e4m3", seed=n + dim)
    j = 1
    for b in (0, 2):
        rows = slice(int(p.starts[b]), int(p.starts[b + 1]))
        p.mask[rows] &= ~np.uint64(1 << j)
        p.mask[rows.start + j] |= np.uint64(1 << j)
        pos = p.ctx[b] + j
        p.v_scale[p.table[b, pos // 16], :, pos % 16] = 2.0 ** huge
    _check(p, few)


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("n", [3, 7, 15])
@pytest.mark.parametrize("at", [0, 1000])   # in the first tile, and later
def test_scale_of_a_position_without_weight(at, n, few):
    """A cached position with a value scale of 2^40 whose score lies about 100 below every row's others:
    its weight, e^-100 = 2^-144, is nothing even so."""
    p = Pass([3000, 5], [n, 2], 8, 2, 128, 16, "e4m3", seed=n)
    p.q[..., 0] = 12.0
    key = torch.zeros(128)
    key[0] = -100.0   # a score of -12 * 100 / sqrt(128) = -106
    codes, scale = quantise_ref(key[None])
    page, row = p.table[0, at // 16], at % 16
    p.k[page, row], p.k_scale[page, :, row] = codes[0], scale[0]
    p.v_scale[page, :, row] = 2.0 ** 40
    _check(p, few)


@pytest.mark.parametrize("few", [True, False])
def test_weight_and_scale_against_each_other(few):
    """The heaviest weights lie on the smallest values: per position the weight falls by as much as its
    scale rises, so that all of 2^20 in scale counts alike."""
    p = Pass([1200], [4], 8, 2, 128, 16, "e4m3", seed=3)
    p.q[..., 0], length = 8.0, 1204
    rise = np.linspace(0, 20, length)[np.random.default_rng(0).permutation(length)]
    for pos in range(length):
        key = torch.zeros(128)
        key[1:] = 0.1 * torch.randn(127, generator=torch.Generator().manual_seed(pos))
        key[0] = float(-rise[pos] * np.log(2) * 128 ** 0.5 / 8)
        codes, scale = quantise_ref(key[None])
        page, row = p.table[0, pos // 16], pos % 16
        p.k[page, row], p.k_scale[page, :, row] = codes[0], scale[0]
        p.v_scale[page, :, row] = float(2.0 ** (rise[pos] - 8))
    _check(p, few)

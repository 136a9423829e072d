"""Non-finite values of drafted tokens in heads whose channels do not fill whole warps: undivided and
divided among CTAs, on the kernel for few rows and on the one for many."""
import numpy as np
import pytest
import torch

from attn_util import Pass, assert_within, weight_eps
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("divided", [False, True])
@pytest.mark.parametrize("n", [3, 7, 15])   # 12, 28 and 60 rows of a key head
@pytest.mark.parametrize("dim,cache", [(8, "bf16"), (24, "bf16"), (40, "bf16"), (72, "bf16"), (104, "bf16"), (120, "bf16"),
                                       (16, "e4m3"), (48, "e4m3"), (80, "e4m3"), (112, "e4m3")])
def test_bad_values_in_any_head(dim, cache, n, divided, few):
    ctx = 126   # the drafts lie in two tiles
    p = Pass([ctx, 40], [n, 2], 8, 2, dim, 16, cache, seed=dim + n)
    j = 1
    p.mask[n - 1] &= ~np.uint64(1 << j)
    seen = [i for i in range(n) if (int(p.mask[i]) >> j) & 1]
    others = [i for i in range(n + 2) if i not in seen]
    page, row, ch = p.table[0, (ctx + j) // 16], (ctx + j) % 16, dim - 3
    if cache == "e4m3":
        p.v[page, row, :, ch] = 0x7F
    else:
        p.v[page, row, :, ch] = float("nan")
    args = p.device(api)
    if divided:
        table = torch.zeros((2, 2500), dtype=torch.int32)
        table[:, : p.table.shape[1]] = torch.from_numpy(p.table)
        args["page_table"] = table.to(DEV)
    ws = api.tree_attention_workspace(args["cache"], n + 2, 2, 8)
    out, lse = api.tree_attention(**args, max_tokens=n if few else 64, return_lse=True, ws=ws)
    assert api.last_device_error(ws) == 0
    ref, ref_lse, ob, lb = p.reference(weight_eps(p), True)
    assert_within("lse", lse, ref_lse, lb)
    assert_within("out", out[others], ref[others], ob[others])
    o = out[seen].float()
    assert seen and bool(o[..., ch].isnan().all()) and bool(o[..., [c for c in range(dim) if c != ch]].isfinite().all())

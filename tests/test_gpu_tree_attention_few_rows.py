"""The kernel for few rows (max_tokens times the group at most 64) at the masks, values, layouts and
errors where it can go wrong: at 16, 32 and 64 rows of a key head, 64 and 128 channels, both cache
formats.  A group of 4 query heads throughout, so 4, 8 or 16 tokens."""
import numpy as np
import pytest
import torch

from attn_util import Pass, assert_within, quantise_ref, weight_eps
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"

every_form = pytest.mark.parametrize("n,dim,cache", [(n, dim, cache) for n in (4, 8, 16) for dim in (64, 128) for cache in ("bf16", "e4m3")])


def _check(p, scale=None, **over):
    """Against the 64-bit reference, with the exact bound on the tokens: twice, the same bits."""
    args = p.device(api)
    args.update(over)
    ws = api.tree_attention_workspace(args["cache"], p.q.shape[0], len(p.n), p.q.shape[1])
    out, lse = api.tree_attention(**args, scale=scale, max_tokens=max(p.n), return_lse=True, ws=ws)
    ref, ref_lse, ob, lb = p.reference(weight_eps(p), True, scale)
    assert_within("lse", lse, ref_lse, lb)
    assert_within("out", out, ref, ob)
    again, lse2 = api.tree_attention(**args, scale=scale, max_tokens=max(p.n), return_lse=True, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    return out, lse


def _requantise(p):
    (p.k, ks), (p.v, vs) = quantise_ref(p.k.float()), quantise_ref(p.v.float())
    p.k_scale, p.v_scale, p.cache_type = ks.transpose(1, 2).contiguous(), vs.transpose(1, 2).contiguous(), "e4m3"


@every_form
def test_ragged_lengths(n, dim, cache):
    """Lengths around a tile, empty contexts, fewer tokens than the bound, chains and trees."""
    for tree in (False, True):
        _check(Pass([127, 128, 129, 0, 1, 255, 640], [n, 1, n - 1, n, 1, 2, n], 8, 2, dim, 16, cache, tree=tree, seed=n + dim))


@every_form
def test_divided_and_joined(n, dim, cache):
    """The same lengths with a page table that has room for far more: parts of an item on several CTAs."""
    p = Pass([2000, 128 - n, 0, 900], [n, n, 3, 1], 8, 2, dim, 16, cache, seed=n)
    table = torch.full((4, 2500), 2 ** 30, dtype=torch.int32)   # unused places may hold anything
    table[:, : p.table.shape[1]] = torch.from_numpy(p.table)
    _check(p, page_table=table.to(DEV))


@every_form
def test_peaked_scores(n, dim, cache):
    """Scores spread over hundreds: one position takes nearly all of a row, far below the others."""
    _check(Pass([900, 40], [n, 2], 8, 2, dim, 32, cache, spread=40.0, seed=3), scale=0.3)


@every_form
@pytest.mark.parametrize("falling", [False, True])
def test_scores_that_rise_or_fall(falling, n, dim, cache):
    """Keys sorted so that the running maxima grow by a few units a tile, or are the first tile's."""
    p = Pass([1500], [n], 8, 2, dim, 16, "bf16", seed=5)
    length = 1500 + n
    ramp = np.linspace(1, 10, length) if not falling else np.linspace(10, 1, length)
    for h in range(2):
        u = p.q[:, h * 4].float().mean(0)
        for pos in range(length):
            p.k[p.table[0, pos // 16], pos % 16, h] = (u * float(ramp[pos]) / u.norm() * 4).to(torch.bfloat16)
    if cache == "e4m3":
        _requantise(p)
    _check(p)


@pytest.mark.parametrize("n", [4, 8, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_values_with_scales_far_apart(dim, n):
    """Value scales over 60 binary orders, small first and last."""
    p = Pass([700], [n], 8, 2, dim, 16, "e4m3", seed=6)
    order = np.linspace(-30, 30, 700 + n)
    for pos in range(700 + n):
        p.v_scale[p.table[0, pos // 16], :, pos % 16] = float(2.0 ** (order[pos] if pos < 600 else -20))
    _check(p)


@every_form
def test_rows_that_see_nothing(n, dim, cache):
    """Empty masks: alone in a context of nothing, beside rows that see something, over a whole sequence;
    and sequences without tokens, and q rows beyond the last sequence, where nothing is written."""
    p = Pass([0, 50, 0, 20], [n, 3, 2, 0], 8, 2, dim, 16, cache, seed=7)
    empty = [1, n - 1, n + 3, n + 4]
    p.mask[empty] = 0
    out, lse = _check(p)
    assert not bool(out[empty].any()) and bool((lse[empty] == -np.inf).all())
    args, total = p.device(api), n + 5
    pad = torch.zeros((total + 2, 8, dim), dtype=torch.bfloat16, device=DEV)
    pad[:total] = args["q"]
    args["q"], args["mask"] = pad, torch.cat([args["mask"], torch.zeros(2, dtype=torch.int64, device=DEV)])
    o2, l2 = torch.full_like(pad, 3.0), torch.full((total + 2, 8), 3.0, device=DEV)
    api.tree_attention(**args, max_tokens=n, out=o2, lse=l2)
    assert torch.equal(o2[:total], out) and torch.equal(l2[:total], lse)
    assert bool((o2[total:] == 3).all()) and bool((l2[total:] == 3).all())


def _bad_draft(p, n, ctx, j):
    """Sequence 0's rows that see drafted token j (never the last), and the others."""
    p.mask[n - 1] &= ~np.uint64(1 << j)
    sees = [bool((int(p.mask[i]) >> j) & 1) for i in range(n)]
    total = p.q.shape[0]
    return [i for i in range(n) if sees[i]], [i for i in range(total) if not (i < n and sees[i])]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx", [100, 126, 1000])   # the draft within a tile, over two tiles, in a later one
@pytest.mark.parametrize("n,dim", [(4, 64), (8, 64), (16, 64), (4, 128), (8, 128), (16, 128)])
def test_masked_places_may_hold_anything(n, dim, ctx, bad):
    p = Pass([ctx, 60], [n, 3], 8, 2, dim, 32, "bf16", seed=9)
    for b in range(2):   # beyond the length
        length = p.ctx[b] + p.n[b]
        pg = p.table[b, (length - 1) // 32]
        p.k[pg, (length - 1) % 32 + 1:] = bad
        p.v[pg, (length - 1) % 32 + 1:] = bad
    j = 2
    seen, others = _bad_draft(p, n, ctx, j)
    pos = ctx + j
    page, row = p.table[0, pos // 32], pos % 32
    p.v[page, row, :, 3] = bad
    out, lse = api.tree_attention(**p.device(api), max_tokens=n, return_lse=True)
    ref, ref_lse, ob, lb = p.reference(weight_eps(p), True)
    assert_within("lse", lse, ref_lse, lb)
    assert_within("out", out[others], ref[others], ob[others])
    o = out[seen].float()
    assert seen and bool(o[..., [c for c in range(dim) if c != 3]].isfinite().all())
    assert bool(o[..., 3].isnan().all()) if bad != bad else bool((o[..., 3] == bad).all())
    p.v[page, row, :, 3] = 0.0
    p.k[page, row] = float("nan")
    ref, ref_lse, ob, lb = p.reference(weight_eps(p), True)
    out, lse = api.tree_attention(**p.device(api), max_tokens=n, return_lse=True)
    assert_within("out", out[others], ref[others], ob[others])
    assert_within("lse", lse[others], ref_lse[others], lb[others])
    assert bool(out[seen].isnan().all())


@pytest.mark.parametrize("ctx", [100, 126, 1000])
@pytest.mark.parametrize("n,dim", [(4, 64), (8, 64), (16, 64), (4, 128), (8, 128), (16, 128)])
def test_masked_places_of_a_quantised_cache(n, dim, ctx):
    p = Pass([ctx, 60], [n, 3], 8, 2, dim, 32, "e4m3", seed=10)
    for b in range(2):
        length = p.ctx[b] + p.n[b]
        pg, after = p.table[b, (length - 1) // 32], (length - 1) % 32 + 1
        p.k[pg, after:], p.v[pg, after:] = 0x7F, 0xFF
        p.k_scale[pg, :, after:], p.v_scale[pg, :, after:] = float("nan"), float("inf")
    j = 2
    seen, others = _bad_draft(p, n, ctx, j)
    pos = ctx + j
    page, row = p.table[0, pos // 32], pos % 32
    p.v[page, row, :, 3] = 0x7F
    ref, _, ob, _ = p.reference(weight_eps(p), True)
    out = api.tree_attention(**p.device(api), max_tokens=n)
    assert_within("out", out[others], ref[others], ob[others])
    o = out[seen].float()
    assert bool(o[..., 3].isnan().all()) and bool(o[..., [c for c in range(dim) if c != 3]].isfinite().all())
    for scale in (float("nan"), float("inf")):
        p.v_scale[page, :, row] = p.k_scale[page, :, row] = scale
        out = api.tree_attention(**p.device(api), max_tokens=n)
        assert_within("out", out[others], ref[others], ob[others])
        assert bool(out[seen][..., 3].isnan().all())


@every_form
def test_strides_streams_and_offsets(n, dim, cache):
    """A heads-major cache, q and out slices of wider rows, a side stream; then pages whose offsets pass
    32 bits: the bits of the plain layout."""
    p = Pass([90, 400], [n, 2], 8, 2, dim, 16, cache, seed=11)
    args = p.device(api)
    base, base_lse = api.tree_attention(**args, max_tokens=n, return_lse=True)
    c, total = args["cache"], n + 2
    hm = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.k, c.v)]
    wide, outw = (torch.zeros((total, 12, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    wide[:, 2:10] = args["q"]
    ws = api.tree_attention_workspace(c, total, 2, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = dict(args, cache=api.KVCache(*hm, c.k_scale, c.v_scale), q=wide[:, 2:10])
        _, lse = api.tree_attention(**other, max_tokens=n, out=outw[:, 2:10], return_lse=True, ws=ws)
    side.synchronize()
    assert torch.equal(outw[:, 2:10], base) and torch.equal(lse, base_lse)
    assert not bool(outw[:, :2].any()) and not bool(outw[:, 10:].any())
    pages, page, heads, _ = c.k.shape
    stride = ((1 << 32) // (pages - 1) + 4096) // 16 * 16
    views = []
    for x in (c.k, c.v):
        big = torch.empty(stride * (pages - 1) + page * heads * dim, dtype=x.dtype, device=DEV)
        views.append(big.as_strided(x.shape, (stride, heads * dim, dim, 1)))
        views[-1].copy_(x)
    far = api.KVCache(*views, c.k_scale, c.v_scale)
    assert torch.equal(api.tree_attention(**dict(args, cache=far), max_tokens=n), base)


@every_form
def test_graph_replay_follows_the_lengths(n, dim, cache):
    p = Pass([90, 400], [n, 2], 8, 2, dim, 16, cache, seed=12)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], n + 2, 2, 8)
    out = torch.empty_like(args["q"])
    api.tree_attention(**args, out=out, ws=ws, max_tokens=n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.tree_attention(**args, out=out, ws=ws, max_tokens=n)
    p.ctx = [13, 250]
    args["ctx"].copy_(torch.tensor(p.ctx, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref, _, ob, _ = p.reference(weight_eps(p), True)
    assert_within("out", out, ref, ob)


@every_form
def test_device_errors(n, dim, cache):
    """A page outside the cache reads as zeros, a sequence that does not fit is skipped."""
    make = lambda: Pass([90, 400, 30], [n, n - 1, 3], 8, 2, dim, 16, cache, seed=13)
    p, total = make(), 2 * n + 2
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], total, 3, 8)
    base = api.tree_attention(**args, ws=ws, max_tokens=n)
    assert api.last_device_error(ws) == 0
    for ctx in (-1, 100000):
        out = torch.full_like(args["q"], 5.0)
        api.tree_attention(**dict(args, ctx=torch.tensor([90, ctx, 30], dtype=torch.int32, device=DEV)), out=out, ws=ws, max_tokens=n)
        assert api.last_device_error(ws) == 5
        assert torch.equal(out[:n], base[:n]) and torch.equal(out[2 * n - 1:], base[2 * n - 1:]) and bool((out[n:2 * n - 1] == 5).all())
    out = torch.full_like(args["q"], 5.0)
    api.tree_attention(**args, out=out, ws=ws, max_tokens=n - 1)   # one token too many in the first
    assert api.last_device_error(ws) == 5
    ref, _, ob, _ = p.reference(weight_eps(p), True)
    assert bool((out[:n] == 5).all())
    assert_within("out", out[n:], ref[n:], ob[n:])
    q = make()
    q.k[q.table[0, 2]] = 0
    q.v[q.table[0, 2]] = 0
    ref, _, ob, _ = q.reference(weight_eps(q), True)
    for bad in (-3, 10 ** 6):
        table = args["page_table"].clone()
        table[0, 2] = bad
        out = api.tree_attention(**dict(args, page_table=table), ws=ws, max_tokens=n)
        assert api.last_device_error(ws) == 5
        assert torch.equal(out[n:], base[n:])
        assert_within("out", out, ref, ob)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,dim,ctx", [(1, 128, 200), (4, 128, 9000), (8, 64, 9000), (8, 128, 300), (16, 128, 9000), (16, 64, 200)])
def test_wait_that_runs_out(n, dim, ctx, cache):
    """With a limit of half a microsecond the call gives up and says so, or, where the barriers' hardware
    waits outlast the limit, has its ordinary results; the next call on the same workspace has them in any
    case."""
    p = Pass([ctx, ctx // 3, ctx // 2], [n] * 3, 32, 8, dim, 64, cache, seed=21)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], p.q.shape[0], 3, 32)
    base = api.tree_attention(**args, ws=ws, max_tokens=n)
    assert api.last_device_error(ws) == 0
    try:
        api.set_wait_limit(1000)
        out = api.tree_attention(**args, ws=ws, max_tokens=n)
        code = api.last_device_error(ws)   # synchronises
    finally:
        api.set_wait_limit(0)
    assert code == 6 or (code == 0 and torch.equal(out, base))
    for _ in range(2):
        assert torch.equal(api.tree_attention(**args, ws=ws, max_tokens=n), base)
        assert api.last_device_error(ws) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,dim", [(4, 64), (8, 64), (16, 64), (4, 128), (8, 128), (16, 128)])
def test_every_cta_walks_many_tiles(n, dim, cache):
    """Long ragged contexts over many heads: tens of tiles a CTA through the rings, several items in turn."""
    p = Pass([9001, 4000, 6500, 130, 7777], [n, 1, n, n, n - 1], 32, 8, dim, 64, cache, seed=n)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], int(p.starts[-1]), 5, 32)
    out, lse = api.tree_attention(**args, max_tokens=n, return_lse=True, ws=ws)
    again = api.tree_attention(**args, max_tokens=n, ws=ws)
    assert api.last_device_error(ws) == 0 and torch.equal(out, again)
    heads = [3, 17]
    full = p.reference_heads(heads, weight_eps(p), True)
    for h in heads:
        assert_within(f"lse {h}", lse[:, h], full[h][1], full[h][3])
        assert_within(f"out {h}", out[:, h], full[h][0], full[h][2])

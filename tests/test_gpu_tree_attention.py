"""Tree attention on the GPU against the 64-bit softmax: chains and trees, ragged contexts, shared
heads, page sizes that end inside a tile, both cache formats, empty rows, what masked places may
hold, strides, streams, long offsets and the device-side errors."""
import numpy as np
import pytest
import torch

from attn_util import E4M3, Pass, assert_within, weight_eps
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _check(p, scale=None, eps=None, **over):
    args = p.device(api)
    args.update(over)
    out, lse = api.tree_attention(**args, scale=scale, return_lse=True)
    bf = p.q.dtype == torch.bfloat16
    ref, ref_lse, ob, lb = p.reference(weight_eps(p) if eps is None else eps, bf, scale)
    assert out.dtype == p.q.dtype
    assert_within("lse", lse, ref_lse, lb)
    assert_within("out", out, ref, ob)
    return out, lse


CASES = [
    # ctx, n, q heads, kv heads, dim, page
    ([0], [1], 4, 4, 128, 16),                                  # one position
    ([300], [1], 32, 4, 128, 16),                               # one token, shared heads
    ([127, 128, 129, 1], [1, 1, 1, 1], 8, 2, 64, 32),           # around a tile
    ([63, 0, 511, 1000], [16, 64, 3, 1], 8, 1, 128, 64),        # ragged trees, more rows than a tile
    ([700], [64], 16, 2, 128, 16),                              # 512 rows of one head
    ([120, 200], [33, 17], 12, 4, 64, 8),                       # a group of 3
    ([250, 90], [20, 7], 64, 1, 128, 128),                      # one cache head for all
    ([97, 513], [9, 40], 6, 6, 96, 24),                         # no sharing, odd dim and page
    ([333], [5], 5, 1, 80, 40),
    ([2500, 0, 77], [4, 2, 12], 16, 4, 128, 256),
    ([4100], [11], 8, 2, 64, 16),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_reference(case, tree, cache):
    ctx, n, hq, hk, dim, page = CASES[case]
    _check(Pass(ctx, n, hq, hk, dim, page, cache, tree=tree, seed=case))


@pytest.mark.parametrize("ctx,n,hq,hk,dim,page,cache", [([40, 0, 129], [3, 20, 1], 4, 2, 64, 16, "f32"), ([70], [9], 2, 1, 256, 5, "f32"),
                                                        ([33], [64], 3, 3, 20, 7, "f32"), ([50, 31], [2, 6], 8, 2, 128, 13, "e4m3")])
def test_fp32_queries(ctx, n, hq, hk, dim, page, cache):
    _check(Pass(ctx, n, hq, hk, dim, page, cache, q_type=torch.float32, seed=dim))


@pytest.mark.parametrize("dim,page,cache", [(256, 16, "bf16"), (128, 20, "bf16"), (192, 32, "e4m3"), (128, 4, "e4m3"), (8, 16, "bf16")])
def test_layouts_off_the_tensor_cores(dim, page, cache):
    """Wide heads and odd page sizes."""
    _check(Pass([150, 3], [7, 12], 8, 2, dim, page, cache, seed=dim + page))


def test_scale_and_peaked_scores():
    """Scores spread over hundreds: one position takes nearly all of a row, far below the others."""
    _check(Pass([900, 40], [6, 30], 8, 2, 128, 32, "bf16", spread=40.0, seed=3), scale=0.3)
    _check(Pass([900, 40], [6, 30], 8, 2, 128, 32, "e4m3", spread=40.0, seed=4), scale=0.3)


def test_rising_scores_keep_earlier_positions():
    """Keys sorted so that every tile raises the running maximum by a few units, and falls after."""
    for cache in ("bf16", "e4m3"):
        p = Pass([1500], [8], 8, 2, 128, 16, "bf16", seed=5)
        ramp = 1 + 9 * np.sin(np.linspace(0, 3.0, 1508))
        for h in range(2):
            u = p.q[:, h * 4].float().mean(0)
            for pos in range(1508):
                p.k[p.table[0, pos // 16], pos % 16, h] = (u * float(ramp[pos]) / u.norm() * 4).to(torch.bfloat16)
        if cache == "e4m3":
            from attn_util import quantise_ref
            (p.k, ks), (p.v, vs) = quantise_ref(p.k.float()), quantise_ref(p.v.float())
            p.k_scale, p.v_scale, p.cache_type = ks.transpose(1, 2).contiguous(), vs.transpose(1, 2).contiguous(), cache
        _check(p)


def test_values_with_scales_far_apart():
    """Value scales over 60 binary orders, small first and last."""
    p = Pass([700], [5], 8, 2, 128, 16, "e4m3", seed=6)
    order = np.linspace(-30, 30, 705)
    for pos in range(705):
        p.v_scale[p.table[0, pos // 16], :, pos % 16] = float(2.0 ** (order[pos] if pos < 600 else -20))
    _check(p)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rows_that_see_nothing(cache):
    p = Pass([0, 50, 0], [6, 3, 2], 8, 2, 128, 16, cache, seed=7)
    p.mask[[1, 4, 9, 10]] = 0
    out, lse = _check(p)
    empty = [1, 4, 9, 10]
    assert not bool(out[empty].any()) and bool((lse[empty] == -np.inf).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_sequences_without_tokens_and_padding_tokens(cache):
    """n_b = 0 and q rows beyond the last sequence: nothing is written there."""
    p = Pass([20, 130, 5], [4, 0, 3], 4, 2, 64, 16, cache, seed=8)
    args = p.device(api)
    pad = torch.zeros((9, 4, 64), dtype=torch.bfloat16, device=DEV)
    pad[:7] = args["q"]
    args["q"], args["mask"] = pad, torch.cat([args["mask"], torch.zeros(2, dtype=torch.int64, device=DEV)])
    out, lse = torch.full_like(pad, 3.0), torch.full((9, 4), 3.0, device=DEV)
    api.tree_attention(**args, out=out, lse=lse)
    ref, ref_lse, ob, lb = p.reference(weight_eps(p), True)
    assert_within("out", out[:7], ref, ob)
    assert bool((out[7:] == 3).all()) and bool((lse[7:] == 3).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_may_hold_anything(bad):
    """Keys and values that a token does not see, and slots beyond the length, hold NaN or
    infinities: rows that do not see them keep their exact values, rows that do get what the
    formula gives."""
    p = Pass([100, 60], [12, 5], 8, 2, 128, 32, "bf16", seed=9)
    clean = p.reference(weight_eps(p), True)
    for b in range(2):   # everything beyond the length, in the last page and the unused ones
        length = p.ctx[b] + p.n[b]
        pg = p.table[b, (length - 1) // 32]
        p.k[pg, (length - 1) % 32 + 1:] = bad
        p.v[pg, (length - 1) % 32 + 1:] = bad
    j = 4   # drafted token 4 of sequence 0
    sees = [bool((int(p.mask[i]) >> j) & 1) for i in range(12)]
    p.mask[11] &= ~np.uint64(1 << j)
    sees[11] = False
    pos = 100 + j
    p.v[p.table[0, pos // 32], pos % 32, :, 3] = bad
    clean = p.reference(weight_eps(p), True)
    args = p.device(api)
    out, lse = api.tree_attention(**args, return_lse=True)
    assert_within("lse", lse, clean[1], clean[3])
    rows = [i for i in range(17) if not (i < 12 and sees[i])]
    assert_within("out", out[rows], clean[0][rows], clean[2][rows])
    seen_rows = [i for i in range(12) if sees[i]]
    o = out[seen_rows].float()
    assert seen_rows and bool(o[..., [c for c in range(128) if c != 3]].isfinite().all())
    assert bool(o[..., 3].isnan().all()) if bad != bad else bool((o[..., 3] == bad).all())
    # a bad key: a masked one is not felt, a seen one makes its rows NaN or the formula's value
    p.v[p.table[0, pos // 32], pos % 32, :, 3] = 0.0
    p.k[p.table[0, pos // 32], pos % 32] = float("nan")
    clean = p.reference(weight_eps(p), True)
    out = api.tree_attention(**p.device(api))
    assert_within("out", out[rows], clean[0][rows], clean[2][rows])
    assert bool(out[seen_rows].isnan().all())


def test_masked_places_of_a_quantised_cache():
    p = Pass([100, 60], [12, 5], 8, 2, 128, 32, "e4m3", seed=10)
    for b in range(2):
        length = p.ctx[b] + p.n[b]
        pg = p.table[b, (length - 1) // 32]
        p.k[pg, (length - 1) % 32 + 1:] = 0x7F
        p.v[pg, (length - 1) % 32 + 1:] = 0xFF
        p.k_scale[pg, :, (length - 1) % 32 + 1:] = float("nan")
        p.v_scale[pg, :, (length - 1) % 32 + 1:] = float("inf")
    j, pos = 4, 104
    p.mask[11] &= ~np.uint64(1 << j)
    sees = [bool((int(p.mask[i]) >> j) & 1) for i in range(12)]
    p.v[p.table[0, pos // 32], pos % 32, :, 3] = 0x7F
    rows = [i for i in range(17) if not (i < 12 and sees[i])]
    seen_rows = [i for i in range(12) if sees[i]]
    clean = p.reference(weight_eps(p), True)
    out = api.tree_attention(**p.device(api))
    assert_within("out", out[rows], clean[0][rows], clean[2][rows])
    assert bool(out[seen_rows][..., 3].isnan().all())
    for scale in (float("nan"), float("inf")):
        p.v_scale[p.table[0, pos // 32], :, pos % 32] = scale
        p.k_scale[p.table[0, pos // 32], :, pos % 32] = scale
        out = api.tree_attention(**p.device(api))
        assert_within("out", out[rows], clean[0][rows], clean[2][rows])
        assert bool(out[seen_rows][..., 3].isnan().all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_strides_streams_and_repeats(cache):
    """q a slice of a projection's output, out a slice too, a heads-major cache, a side stream:
    the same bits as the plain layout, twice."""
    p = Pass([90, 400], [10, 6], 8, 2, 128, 16, cache, seed=11)
    args = p.device(api)
    base, base_lse = api.tree_attention(**args, return_lse=True)
    c = args["cache"]
    hm = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.k, c.v)]
    wide = torch.zeros((16, 12, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10] = args["q"]
    outw = torch.zeros((16, 12, 128), dtype=torch.bfloat16, device=DEV)
    ws = api.tree_attention_workspace(c, 16, 2, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        args.update(cache=api.KVCache(*hm, c.k_scale, c.v_scale), q=wide[:, 2:10])
        for _ in range(2):
            _, lse = api.tree_attention(**args, out=outw[:, 2:10], return_lse=True, ws=ws)
    side.synchronize()
    assert torch.equal(outw[:, 2:10], base) and torch.equal(lse, base_lse)
    assert not bool(outw[:, :2].any()) and not bool(outw[:, 10:].any())
    assert api.last_device_error(ws) == 0


def test_cuda_graph_replay_follows_the_lengths():
    """Lengths and tables are read on the device: one captured call serves new ones."""
    p = Pass([90, 400], [10, 6], 8, 2, 128, 16, "bf16", seed=12)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], 16, 2, 8)
    out = torch.empty_like(args["q"])
    api.tree_attention(**args, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.tree_attention(**args, out=out, ws=ws)
    p.ctx = [13, 250]
    args["ctx"].copy_(torch.tensor(p.ctx, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref, _, ob, _ = p.reference(weight_eps(p), True)
    assert_within("out", out, ref, ob)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_device_errors(cache):
    """A page outside the cache reads as zeros, a sequence that does not fit is skipped; both are
    recorded, and the others keep their results."""
    p = Pass([90, 400, 30], [10, 6, 3], 8, 2, 128, 16, cache, seed=13)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], 19, 3, 8)
    base = api.tree_attention(**args, ws=ws)
    assert api.last_device_error(ws) == 0
    for ctx in (-1, 100000):
        a = dict(args, ctx=torch.tensor([90, ctx, 30], dtype=torch.int32, device=DEV))
        out = torch.full_like(args["q"], 5.0)
        api.tree_attention(**a, out=out, ws=ws)
        assert api.last_device_error(ws) == 5
        assert torch.equal(out[:10], base[:10]) and torch.equal(out[16:], base[16:]) and bool((out[10:16] == 5).all())
    out = torch.full_like(args["q"], 5.0)
    api.tree_attention(**args, out=out, ws=ws, max_tokens=6)
    assert api.last_device_error(ws) == 5
    # a smaller bound may run on the kernel for few rows: the others are held to the reference
    ref, _, ob, _ = p.reference(weight_eps(p), True)
    assert bool((out[:10] == 5).all())
    assert_within("out", out[10:], ref[10:], ob[10:])
    for bad in (-3, 10 ** 6):
        table = args["page_table"].clone()
        table[0, 2] = bad
        out = api.tree_attention(**dict(args, page_table=table), ws=ws)
        assert api.last_device_error(ws) == 5
        assert torch.equal(out[10:], base[10:])
        q = Pass([90, 400, 30], [10, 6, 3], 8, 2, 128, 16, cache, seed=13)
        q.k[q.table[0, 2]] = 0
        q.v[q.table[0, 2]] = 0
        ref, _, ob, _ = q.reference(weight_eps(q), True)
        assert_within("out", out, ref, ob)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_long_cache_offsets_pass_32_bits(cache):
    p = Pass([60], [3], 4, 1, 128, 16, cache, seed=14, spare=1)
    base = api.tree_attention(**p.device(api))
    pages, page, heads, dim = p.k.shape
    stride = ((1 << 32) // (pages - 1) + 4096) // 16 * 16
    args = p.device(api)
    views = []
    for x in (args["cache"].k, args["cache"].v):
        big = torch.empty(stride * (pages - 1) + page * heads * dim, dtype=x.dtype, device=DEV)
        v = big.as_strided(x.shape, (stride, heads * dim, dim, 1))
        v.copy_(x)
        views.append(v)
    args["cache"] = api.KVCache(*views, args["cache"].k_scale, args["cache"].v_scale)
    assert torch.equal(api.tree_attention(**args), base)


def test_long_context():
    """A context of 40,000 positions: many splits of one row."""
    for cache in ("bf16", "e4m3"):
        _check(Pass([40001], [3], 2, 1, 128, 64, cache, seed=15))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,dim", [(2, 128), (7, 128), (15, 128), (2, 64), (14, 64), (30, 128), (64, 64)])
def test_every_cta_walks_many_tiles(n, dim, cache):
    """Long ragged contexts over many heads: each CTA streams tens of tiles through its rings and
    crosses from one item to the next, with odd tile counts, on both kernels and every row width."""
    ctx = [9001, 4000, 6500, 130, 7777]
    p = Pass(ctx, [n, 1, n, n, max(1, n - 1)], 32, 8, dim, 64, cache, seed=n)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], int(p.starts[-1]), 5, 32)
    out, lse = api.tree_attention(**args, max_tokens=n, return_lse=True, ws=ws)
    again = api.tree_attention(**args, max_tokens=n, ws=ws)
    assert api.last_device_error(ws) == 0
    assert torch.equal(out, again)
    heads = [0, 5, 31]   # the reference of every eighth cache head or so
    full = p.reference_heads(heads, weight_eps(p), True)
    for h in heads:
        assert_within(f"lse {h}", lse[:, h], full[h][1], full[h][3])
        assert_within(f"out {h}", out[:, h], full[h][0], full[h][2])


def test_empty_call():
    c = api.kv_cache(1, 16, 2, 64)
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = api.tree_attention(c, e, z, torch.empty(0, dtype=torch.int32, device=DEV), torch.empty((0, 1), dtype=torch.int32, device=DEV))
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_wide_page_tables(case, cache):
    """A table with room for far longer contexts than these: the same lengths are then divided among
    CTAs and joined, where a table of just their width leaves short ones whole."""
    ctx, n, hq, hk, dim, page = CASES[case]
    p = Pass(ctx, n, hq, hk, dim, page, cache, tree=True, seed=case)
    table = torch.from_numpy(p.table)
    wide = torch.full((table.shape[0], 40000 // page), 2 ** 30, dtype=torch.int32)   # unused places may hold anything
    wide[:, : table.shape[1]] = table
    _check(p, page_table=wide.to(DEV))
    narrow = p.device(api)
    ws = api.tree_attention_workspace(narrow["cache"], p.q.shape[0], len(ctx), hq)
    api.tree_attention(**dict(narrow, page_table=wide.to(DEV)), ws=ws)
    assert api.last_device_error(ws) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,n", [([9000, 300, 4000], 4), ([9000, 300, 4000], 16), ([6000, 5000], 64), ([200, 100], 8)])
def test_wait_that_runs_out_reports_timeout(ctx, n, cache):
    """With a limit of half a microsecond the call gives up and says so, or, where the barriers'
    hardware waits outlast the limit (they return when the data are there), has its ordinary results;
    the next call on the same workspace has them in any case.  V's cleaner polls a count in shared
    memory: over a long bf16 cache its wait for a part's last tile is always beyond the limit."""
    p = Pass(ctx, [n] * len(ctx), 32, 8, 128, 64, cache, seed=21)
    args = p.device(api)
    ws = api.tree_attention_workspace(args["cache"], p.q.shape[0], len(ctx), 32)
    base = api.tree_attention(**args, ws=ws)
    assert api.last_device_error(ws) == 0
    try:
        api.set_wait_limit(1000)
        out = api.tree_attention(**args, ws=ws)
        code = api.last_device_error(ws)   # synchronises
    finally:
        api.set_wait_limit(0)
    if cache == "bf16" and ctx[0] > 4000:
        assert code == 6   # MOE_ERR_DEVICE_TIMEOUT
    assert code == 6 or (code == 0 and torch.equal(out, base))
    for _ in range(2):
        assert torch.equal(api.tree_attention(**args, ws=ws), base)
        assert api.last_device_error(ws) == 0

"""Latent cache rows and latent attention against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from attn_util import rotate_bound, rotate_ref
from latent_util import LatentPass, within
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def run(p, **kw):
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], p.q.shape[0], len(p.n), p.heads)
    out, lse = api.latent_attention(**d, return_lse=True, ws=ws, **{"max_tokens": max(1, max(p.n)), **kw})
    assert api.last_device_error(ws) == 0
    return out, lse


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("ctx,n,heads,rank,rope,page", [
    ([300], [1], 16, 512, 64, 64),            # one token, one block of 16 rows
    ([0], [1], 16, 512, 64, 64),              # nothing but itself
    ([63, 64, 65], [1, 1, 1], 16, 512, 64, 64),
    ([127, 128, 0, 1], [2, 2, 2, 1], 16, 512, 64, 32),
    ([1000, 17, 450], [4, 3, 1], 16, 512, 64, 64),       # 64 rows
    ([200, 31], [7, 5], 16, 512, 64, 16),                # several blocks, the last part empty
    ([700, 90], [64, 33], 16, 512, 64, 128),
    ([500], [3], 128, 512, 64, 64),
    ([130, 40], [5, 2], 12, 256, 64, 8),
    ([90, 333], [3, 9], 5, 128, 32, 24),
    ([77], [6], 3, 384, 48, 40),
    ([260], [8], 7, 72, 16, 16),
    ([1500] * 3 + [3] * 40, [1] * 43, 8, 512, 64, 64),   # more than 32 sequences
    ([5000, 4999], [4, 4], 16, 512, 64, 64),             # parts of many CTAs
    ([9000], [1], 16, 512, 64, 64),
])
@pytest.mark.parametrize("tree", [False, True])
def test_tensor_cores(ctx, n, heads, rank, rope, page, tree):
    p = LatentPass(ctx, n, heads, rank, rope, page, tree=tree, seed=len(ctx) + heads)
    p.check(api, *run(p))


@pytest.mark.parametrize("kind,q_kind,page,rope", [(F32, F32, 16, 64), (F32, BF16, 16, 64), (BF16, F32, 16, 64), (BF16, BF16, 4, 64),
                                                   (BF16, BF16, 16, 128), (F32, F32, 3, 4)])
@pytest.mark.parametrize("rank", [64, 200, 512])
def test_cuda_cores(kind, q_kind, page, rope, rank):
    p = LatentPass([70, 0, 33], [5, 2, 1], 9, rank, rope, page, kind, q_kind, seed=rank)
    assert not p.on_tensor_cores()
    p.check(api, *run(p))


@pytest.mark.parametrize("ctx,n", [([2000, 5, 0], [3, 2, 1]), ([4000], [1]), ([700] * 9, [8] * 9), ([300] * 40, [20] * 40)])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_cuda_cores_divide_the_positions(ctx, n, kind):
    """Parts of many CTAs, parts that are empty, and rows enough for none."""
    p = LatentPass(ctx, n, 5, 72, 8, 6, kind, F32, seed=len(ctx))
    out, lse = run(p)
    p.check(api, out, lse)
    again = run(p)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_cuda_cores_do_not_touch_what_is_not_seen(value):
    p = LatentPass([300, 64], [4, 2], 4, 256, 32, 6, F32, F32, seed=4)
    p.mask[:4] = [1, 2, 5, 0]
    p.mask[4:] = [1, 3]
    page, row = p.at(0, 301)
    p.rows[page, row, 7] = value
    for b in range(2):
        page, row = p.at(b, p.ctx[b] + p.n[b] - 1)
        p.rows[page, row + 1:] = value
    out, lse = run(p)
    assert not torch.isfinite(out[1, :, 7]).any()
    keep = [0, 2, 3, 4, 5]
    ref, ref_lse, bound, lse_bound = p.reference(0.0, False)
    within("out", out[keep], ref[keep], bound[keep])
    within("lse", lse[keep], ref_lse[keep], lse_bound[keep])


@pytest.mark.parametrize("heads", [4, 8, 16])   # blocks of 16, 32 and 64 rows
def test_rows_that_see_nothing(heads):
    p = LatentPass([0, 150], [4, 3], heads, 512, 64, 64, seed=3)
    p.mask[0] = p.mask[2] = 0    # of the sequence without a context
    p.mask[5] = 0                # sees its context
    out, lse = run(p)
    assert out[0].eq(0).all() and out[2].eq(0).all() and lse[0].eq(-np.inf).all() and lse[2].eq(-np.inf).all()
    p.check(api, out, lse)


@pytest.mark.parametrize("heads", [4, 8, 16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), torch.finfo(BF16).min])
def test_what_is_not_seen_does_not_count(heads, value):
    """Non-finite rows of drafted tokens reach only those that see them; what lies beyond the length
    reaches nobody."""
    p = LatentPass([130, 64], [4, 2], heads, 512, 64, 64, seed=4)
    p.mask[:4] = [1, 2, 5, 8]            # token 1 is seen by itself alone
    p.mask[4:] = [1, 3]
    page, row = p.at(0, 131)
    p.rows[page, row, 7] = value
    for b in range(2):                    # behind the last token, to the end of its page
        page, row = p.at(b, p.ctx[b] + p.n[b] - 1)
        p.rows[page, row + 1:] = value
    out, lse = run(p)
    if not np.isfinite(value):
        assert not torch.isfinite(out[1, :, 7]).any()
    keep = [0, 2, 3, 4, 5]
    ref, ref_lse, bound, lse_bound = p.reference(2.0 ** -8, True)
    within("out", out[keep], ref[keep], bound[keep])
    within("lse", lse[keep], ref_lse[keep], lse_bound[keep])


def test_a_cached_value_is_every_rows():
    p = LatentPass([100], [3], 16, 512, 64, 64, seed=5)
    page, row = p.at(0, 20)
    p.rows[page, row, 3] = float("nan")
    out, lse = run(p)
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("heads", [4, 16])
def test_growing_scores(heads):
    """Maxima that grow from tile to tile by far more than the bound for leaving the output as it is."""
    p = LatentPass([700], [4], heads, 512, 64, 64, seed=6, spread=0.2)
    q = p.q[:, :, :1].float().abs() + 1
    p.q[:, :, 0] = q[:, :, 0].to(BF16)
    place = np.array([p.at(0, i) for i in range(704)])
    p.rows[place[:, 0], place[:, 1], 0] = torch.linspace(-2000, 2000, 704).to(BF16)
    p.check(api, *run(p))


def test_repeats_and_bounds_are_alike():
    p = LatentPass([3000, 700, 45], [3, 1, 4], 16, 512, 64, 64, seed=7)
    out, lse = run(p)
    for _ in range(3):
        again = run(p)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    p.check(api, *run(p, max_tokens=64))   # a loose bound


def test_strides_and_views():
    p = LatentPass([200, 90], [3, 2], 16, 512, 64, 32, seed=8)
    d = p.device(api)
    wide = torch.full((p.rows.shape[0], 40, 640), float("nan"), dtype=BF16, device="cuda")
    wide[:, :32, :576] = d["cache"].rows
    d["cache"] = api.LatentCache(wide[:, :32, :576], 512)
    q = torch.full((5, 18, 640), float("nan"), dtype=BF16, device="cuda")
    q[:, 1:17, 8:584] = d["q"]
    out = torch.full((5, 20, 520), 7.0, dtype=BF16, device="cuda")
    lse = torch.empty((5, 16), device="cuda")
    d["q"] = q[:, 1:17, 8:584]
    api.latent_attention(**d, out=out[:, 2:18, :512], lse=lse, max_tokens=3)
    p.check(api, out[:, 2:18, :512], lse)
    out[:, 2:18, :512] = 7.0
    assert out.eq(7.0).all()
    # addresses that 16-byte accesses do not take: the CUDA cores
    odd = torch.zeros((5, 16, 577), dtype=BF16, device="cuda")
    odd[..., 1:] = q[:, 1:17, 8:584]
    d["q"] = odd[..., 1:]
    out2, lse2 = api.latent_attention(**d, return_lse=True, max_tokens=3)
    p.check(api, out2, lse2)


def test_bad_lengths_and_pages_are_recorded():
    p = LatentPass([100, 100, 100], [2, 2, 2], 16, 512, 64, 64, seed=9)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 6, 3, 16)
    d["ctx"][1] = 10 ** 6
    out = torch.full((6, 16, 512), 3.0, dtype=BF16, device="cuda")
    lse = torch.full((6, 16), 3.0, device="cuda")
    api.latent_attention(**d, out=out, lse=lse, ws=ws, max_tokens=2)
    assert api.last_device_error(ws) == 5
    assert out[2:4].eq(3.0).all() and lse[2:4].eq(3.0).all()
    keep = [0, 1, 4, 5]
    ref, ref_lse, bound, lse_bound = p.reference(2.0 ** -8, True)
    within("out", out[keep], ref[keep], bound[keep])
    within("lse", lse[keep], ref_lse[keep], lse_bound[keep])
    # a page outside the cache reads as zeros
    d = p.device(api)
    d["page_table"][0, 0] = p.rows.shape[0]
    p.rows = torch.cat([p.rows, torch.zeros_like(p.rows[:1])])
    p.table[0, 0] = p.rows.shape[0] - 1
    out, lse = api.latent_attention(**d, return_lse=True, ws=ws, max_tokens=2)
    assert api.last_device_error(ws) == 5
    p.check(api, out, lse)


def test_page_numbers_of_any_kind():
    """Negative ones and large ones read as zeros, the smallest integers among them."""
    for odd in (-1, -2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1):
        p = LatentPass([200], [2], 16, 512, 64, 16, seed=13)
        d = p.device(api)
        ws = api.latent_attention_workspace(d["cache"], 2, 1, 16)
        api.latent_attention(**p.device(api), ws=ws, max_tokens=2)   # the ring holds other rows
        assert api.last_device_error(ws) == 0
        d["page_table"][0, 5] = odd
        p.rows = torch.cat([p.rows, torch.zeros_like(p.rows[:1])])
        p.table[0, 5] = p.rows.shape[0] - 1
        out, lse = api.latent_attention(**d, return_lse=True, ws=ws, max_tokens=2)
        assert api.last_device_error(ws) == 5
        p.check(api, out, lse)


def test_rows_behind_the_last_sequence_and_other_orders():
    p = LatentPass([300, 70], [3, 2], 16, 512, 64, 32, seed=14)
    d = p.device(api)
    ref = api.latent_attention(**d, return_lse=True, max_tokens=3)
    # tokens that no sequence has
    more = torch.cat([d["q"], torch.full((3, 16, 576), float("nan"), dtype=BF16, device="cuda")])
    out, lse = torch.full((8, 16, 512), 5.0, dtype=BF16, device="cuda"), torch.full((8, 16), 5.0, device="cuda")
    api.latent_attention(**{**d, "q": more, "mask": torch.cat([d["mask"], d["mask"][:3]])}, out=out, lse=lse, max_tokens=3)
    assert torch.equal(out[:5], ref[0]) and torch.equal(lse[:5], ref[1]) and out[5:].eq(5.0).all() and lse[5:].eq(5.0).all()
    # heads outside tokens, in what is read and what is written
    q = d["q"].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((16, 5, 512), dtype=BF16, device="cuda").transpose(0, 1)
    api.latent_attention(**{**d, "q": q}, out=out, lse=lse[:5], max_tokens=3)
    assert torch.equal(out, ref[0]) and torch.equal(lse[:5], ref[1])


def test_two_streams_at_once():
    a, b = LatentPass([5000, 100], [4, 2], 16, 512, 64, 64, seed=15), LatentPass([4000] * 3, [1] * 3, 16, 512, 64, 64, seed=16)
    da, db = a.device(api), b.device(api)
    wa, wb = api.latent_attention_workspace(da["cache"], 6, 2, 16), api.latent_attention_workspace(db["cache"], 3, 3, 16)
    ra, rb = (api.latent_attention(**x, ws=w, max_tokens=4) for x, w in ((da, wa), (db, wb)))
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        for s, x, w in ((sa, da, wa), (sb, db, wb)):
            with torch.cuda.stream(s):
                got.append(api.latent_attention(**x, ws=w, max_tokens=4))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) for x in got[::2]) and all(torch.equal(x, rb) for x in got[1::2])
    assert api.last_device_error(wa) == 0 and api.last_device_error(wb) == 0


def test_empty_sequences():
    p = LatentPass([50, 70, 20], [2, 0, 1], 16, 512, 64, 64, seed=10)
    p.check(api, *run(p))
    d = LatentPass([50], [0], 16, 512, 64, 64).device(api)
    assert api.latent_attention(**d).shape == (0, 16, 512)


def test_graph_and_stream():
    p = LatentPass([4000, 300], [2, 4], 16, 512, 64, 64, seed=11)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 6, 2, 16)
    out, lse = torch.zeros((6, 16, 512), dtype=BF16, device="cuda"), torch.zeros((6, 16), device="cuda")
    call = lambda: api.latent_attention(**d, out=out, lse=lse, ws=ws, max_tokens=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    out.zero_()
    lse.zero_()
    graph.replay()
    p.check(api, out, lse)
    # other lengths in the same memory
    d["ctx"].copy_(torch.tensor([100, 17], dtype=torch.int32))
    p.ctx = [100, 17]
    graph.replay()
    p.check(api, out, lse)
    assert api.last_device_error(ws) == 0


@pytest.mark.parametrize("heads", [4, 8, 16])
def test_wait_that_runs_out(heads):
    """With a limit of half a microsecond the call gives up and says so, or, where the barriers' hardware waits
    outlast the limit (they return when the data are there), has its ordinary results; the next call on
    the same workspace has them in any case."""
    p = LatentPass([9000, 300], [4, 4], heads, 512, 64, 64, seed=12)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 8, 2, heads)
    base = api.latent_attention(**d, ws=ws, max_tokens=4)
    assert api.last_device_error(ws) == 0
    for limit in (1, 1000):
        api.set_wait_limit(limit)
        try:
            out = api.latent_attention(**d, ws=ws, max_tokens=4)
            code = api.last_device_error(ws)   # synchronises
        finally:
            api.set_wait_limit(0)
        assert code == 6 or (code == 0 and torch.equal(out, base))
        assert torch.equal(api.latent_attention(**d, ws=ws, max_tokens=4), base)
        assert api.last_device_error(ws) == 0


# ---------------------------------------------------------------- rows
def write_case(tokens, heads, rank, rope, rot, kind, cache_kind, page, interleaved, norm, seed):
    g = torch.Generator().manual_seed(seed)
    w, mag = 1e4 ** (-2.0 * np.arange(rot // 2) / rot), 1.0
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:tokens].int()
    if tokens > 3:
        slots[1] = -1
    return dict(latent=torch.randn((tokens, rank), generator=g).to(kind), k=torch.randn((tokens, rope), generator=g).to(kind),
                q=torch.randn((tokens, heads, rope), generator=g).to(kind), norm=torch.rand(rank, generator=g) + 0.5 if norm else None,
                slots=slots, positions=torch.randint(0, 5000, (tokens,), generator=g).int(), w=w,
                rows=torch.randn((pages, page, rank + rope), generator=g).to(cache_kind), interleaved=interleaved)


@pytest.mark.parametrize("tokens,heads,rank,rope,rot,page", [(1, 16, 512, 64, 64, 64), (37, 33, 512, 64, 64, 16), (5, 7, 256, 32, 32, 8),
                                                              (9, 3, 64, 128, 64, 24), (6, 2, 504, 48, 16, 5), (4, 3, 72, 24, 22, 7)])
@pytest.mark.parametrize("kind,cache_kind", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("interleaved,norm", [(True, True), (False, True), (True, False)])
def test_write(tokens, heads, rank, rope, rot, page, kind, cache_kind, interleaved, norm):
    c = write_case(tokens, heads, rank, rope, rot, kind, cache_kind, page, interleaved, norm, rank + tokens)
    rows = c["rows"].cuda()
    cache = api.LatentCache(rows, rank)
    table = api.rope_table(5000, c["w"])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    n = None if c["norm"] is None else c["norm"].cuda()
    q = api.latent_write(cache, c["latent"].cuda(), c["k"].cuda(), c["slots"].cuda(), norm=n, eps=1e-5, q=c["q"].cuda(),
                         positions=c["positions"].cuda(), table=table, interleaved=interleaved, ws=ws)
    assert api.last_device_error(ws) == 0
    x = c["latent"].double()
    if norm:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * c["norm"].double()
    # mean of squares in fp32 to (rank + 2) 2^-24, halved by the root, root, quotient and two products 2^-24 each
    e = (0.5 * (rank + 2) + 5) * 2.0 ** -24 * x.abs() * (1 if norm else 0)
    if cache_kind == BF16:
        e = e + 2.0 ** -8 * (x.abs() + e)
    turned = torch.from_numpy(rotate_ref(c["k"][:, None].double().numpy(), c["positions"].numpy(), c["w"], 1.0, rot, interleaved))
    bound = torch.as_tensor(rotate_bound(c["k"][:, None].double().numpy(), c["w"], 1.0, rot, interleaved, cache_kind == BF16, turned.numpy()))
    ref, limit = c["rows"].double(), torch.zeros_like(c["rows"].double())
    for t, slot in enumerate(c["slots"].tolist()):
        if slot >= 0:
            ref[slot // page, slot % page] = torch.cat((x[t], turned[t, 0]))
            limit[slot // page, slot % page] = torch.cat((e[t], bound[t, 0]))
    within("rows", rows, ref, limit)
    turned = torch.from_numpy(rotate_ref(c["q"].double().numpy(), c["positions"].numpy(), c["w"], 1.0, rot, interleaved))
    within("q", q, turned, torch.as_tensor(rotate_bound(c["q"].double().numpy(), c["w"], 1.0, rot, interleaved, kind == BF16, turned.numpy())))


def test_write_views_in_place_and_out_of_range():
    c = write_case(6, 4, 512, 64, 64, BF16, BF16, 16, True, False, 1)
    table = api.rope_table(5000, c["w"])
    plain = c["rows"].cuda()
    q0 = api.latent_write(api.LatentCache(plain, 512), c["latent"].cuda(), c["k"].cuda(), c["slots"].cuda(), q=c["q"].cuda(),
                          positions=c["positions"].cuda(), table=table, interleaved=True)
    both = torch.cat((c["latent"], c["k"]), 1).cuda()
    q = torch.zeros((6, 4, 200), dtype=BF16, device="cuda")
    q[..., 136:] = c["q"].cuda()
    rows = c["rows"].cuda()
    got = api.latent_write(api.LatentCache(rows, 512), both[:, :512], both[:, 512:], c["slots"].cuda(), q=q[..., 136:],
                           positions=c["positions"].cuda(), table=table, interleaved=True, q_out=q[..., 136:])
    assert torch.equal(rows, plain) and torch.equal(q[..., 136:], q0) and got.data_ptr() == q[..., 136:].data_ptr()
    # the kernel for any layout: the same bits without a norm
    odd = torch.zeros((6, 577), dtype=BF16, device="cuda")
    odd[:, 1:] = both
    rows = c["rows"].cuda()
    q2 = api.latent_write(api.LatentCache(rows, 512), odd[:, 1:513], odd[:, 513:], c["slots"].cuda(), q=c["q"].cuda(),
                          positions=c["positions"].cuda(), table=table, interleaved=True)
    assert torch.equal(rows, plain) and torch.equal(q2, q0)
    # a slot and a position out of range take nothing and are recorded
    for odd_layout in (False, True):
        slots, positions, rows, ws = c["slots"].cuda(), c["positions"].cuda(), c["rows"].cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
        slots[0], positions[2] = rows.shape[0] * 16, 5000
        q_out = torch.full_like(q0, 9.0)
        src = odd[:, 1:] if odd_layout else both
        api.latent_write(api.LatentCache(rows, 512), src[:, :512], src[:, 512:], slots, q=c["q"].cuda(), positions=positions,
                         table=table, interleaved=True, q_out=q_out, ws=ws)
        assert api.last_device_error(ws) == 5
        want = plain.clone()
        for t in (0, 2):
            s = int(c["slots"][t])
            want[s // 16, s % 16] = c["rows"].cuda()[s // 16, s % 16]
        assert torch.equal(rows, want) and q_out[2].eq(9.0).all() and torch.equal(q_out[3], q0[3])


def test_write_without_rotation():
    c = write_case(5, 1, 128, 32, 32, BF16, BF16, 8, False, False, 2)
    rows = c["rows"].cuda()
    assert api.latent_write(api.LatentCache(rows, 128), c["latent"].cuda(), c["k"].cuda(), c["slots"].cuda()) is None
    for t, s in enumerate(c["slots"].tolist()):
        if s >= 0:
            assert torch.equal(rows[s // 8, s % 8].cpu(), torch.cat((c["latent"][t], c["k"][t])))


def test_absorbed_form_is_attention_with_expanded_heads():
    """Queries times key matrices, then outputs times value matrices, against attention with each head's
    own keys and values in 64 bits."""
    g = torch.Generator().manual_seed(3)
    heads, nope, value, rank, rope, ctx, n, page = 4, 32, 48, 128, 32, 50, 3, 16
    wk, wv = (torch.randn((heads, d, rank), generator=g, dtype=torch.float64) * rank ** -0.5 for d in (nope, value))
    c = torch.randn((ctx + n, rank + rope), generator=g)
    q = torch.randn((n, heads, nope + rope), generator=g)
    cache = api.latent_cache(4, page, rank, rope, "f32")
    api.latent_write(cache, c[:, :rank].cuda(), c[:, rank:].cuda(), torch.arange(ctx + n).int().cuda())
    qa = torch.cat((torch.einsum("nhd,hdr->nhr", q[..., :nope].double(), wk), q[..., nope:].double()), -1).float().cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    scale = (nope + rope) ** -0.5
    out = api.latent_attention(cache, qa, i32(0, n), i32(ctx), i32(0, 1, 2, 3)[None], scale)
    got = torch.einsum("nhr,hvr->nhv", out.double().cpu(), wv)
    k = torch.cat((torch.einsum("pr,hdr->hpd", c[:, :rank].double(), wk), c[:, rank:].double().expand(heads, -1, -1)), -1)
    v = torch.einsum("pr,hvr->hpv", c[:, :rank].double(), wv)
    s = torch.einsum("nhd,hpd->hnp", q.double(), k) * scale
    see = torch.arange(ctx + n) <= ctx + torch.arange(n)[:, None]
    want = torch.einsum("hnp,hpv->nhv", torch.softmax(s.masked_fill(~see, -np.inf), -1), v)
    # fp32 throughout: a score off by about 160 roundings of its terms' sum (below 60), twice that in a
    # weight, on outputs of sums below 10
    assert (got - want).abs().max() < 2 * 160 * 2.0 ** -24 * 60 * 10

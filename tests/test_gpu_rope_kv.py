"""Rotary positions and cache rows on the GPU against 64-bit references: every layout, partial
rotation, types, odd sizes and strides, gradients, quantised writes and reads bit for bit, and the
device-side errors."""
import numpy as np
import pytest
import torch

from attn_util import E4M3, assert_within, quantise_ref, rotate_bound, rotate_ref
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _table(rot, positions=4096, scaling="plain", factor=1.0, original=0, base=1e6):
    w, mag = api.rope_frequencies(rot, base=base, scaling=scaling, factor=factor, original=original)
    return w, mag, api.rope_table(positions, w, mag)


def _rows(seed, tokens, heads, dim, dtype):
    return torch.randn((tokens, heads, dim), generator=torch.Generator().manual_seed(seed)).to(dtype)


def test_table_is_the_rounded_double():
    w, mag, table = _table(128, 131072, "by_parts", 4.0, 32768)
    p = np.array([0, 1, 17, 4095, 131071])
    ang = p[:, None] * w[None]
    ref = torch.from_numpy(np.stack([mag * np.cos(ang), mag * np.sin(ang)], -1))
    # rounded to fp32 once; the double sine and cosine are off by a few 2^-53 of the angle at most
    assert_within("table", table[_t(p)], ref, 2.0 ** -24 * ref.abs() + 2.0 ** -52 * 131072)


@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [(1, 32, 4, 128, 128), (37, 8, 8, 64, 64), (5, 6, 2, 128, 64), (9, 3, 1, 96, 96),
                                                  (300, 4, 1, 80, 64), (7, 2, 1, 50, 14), (3, 1, 1, 256, 256), (4, 2, 2, 33, 2),
                                                  (65, 5, 1, 144, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(tokens, hq, hk, dim, rot, interleaved, dtype):
    w, mag, table = _table(rot, scaling="linear", factor=2.5)
    pos = np.random.default_rng(dim).integers(0, 4096, tokens).astype(np.int32)
    q, k = _rows(1, tokens, hq, dim, dtype), _rows(2, tokens, hk, dim, dtype)
    for inverse in (False, True):
        qo, ko = api.rope(q.to(DEV), k.to(DEV), _t(pos), table, interleaved=interleaved, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            x = x.double().numpy()
            ref = rotate_ref(x, pos, w, mag, rot, interleaved, inverse)
            bound = rotate_bound(x, w, mag, rot, interleaved, dtype == torch.bfloat16, ref)
            assert y.dtype == dtype
            assert_within("rope", y, torch.from_numpy(ref), torch.from_numpy(bound))
            assert torch.equal(y.cpu()[..., rot:], torch.from_numpy(x)[..., rot:].to(dtype))


def test_rope_gradient_is_the_transpose_and_matches_differences():
    """<g, R(x)> = <R^T g, x>, and each element of R^T g is the difference quotient of <g, R(x)>.
    R is linear, so a quotient with step 1 in a single channel is exact up to fp32 rounding."""
    tokens, heads, dim, rot = 3, 2, 48, 32
    for interleaved in (False, True):
        w, mag, table = _table(rot, scaling="by_parts", factor=8.0, original=512)
        pos = _t(np.array([3, 700, 4095], np.int32))
        x, g = (_rows(s, tokens, heads, dim, torch.float32).to(DEV) for s in (3, 4))
        fwd = lambda z: api.rope(z, None, pos, table, interleaved=interleaved)[0].double()
        grad = api.rope(g, None, pos, table, interleaved=interleaved, inverse=True)[0].double()
        gd = g.double()
        # every dot product here has tokens * heads * dim terms of size <= ~16, each off by 2^-22
        tol = 2.0 ** -22 * 16 * tokens * heads * dim * mag
        assert abs(float((gd * fwd(x)).sum() - (grad * x.double()).sum())) <= tol
        base = fwd(x)
        for at in [(0, 0, 0), (1, 1, 17), (2, 0, 31), (2, 1, 40), (1, 0, 16)]:
            e = x.clone()
            e[at] += 1.0
            step = float(e[at].double() - x[at].double())
            assert abs(float((gd * (fwd(e) - base)).sum()) / step - float(grad[at])) <= tol


def test_rope_strided_in_place_and_q_only():
    """Views of one projection's output, written back in place; k alone; another stream."""
    w, mag, table = _table(64)
    x = _rows(5, 19, 10, 64, torch.bfloat16)
    pos = np.arange(100, 119, dtype=np.int32)
    ref = rotate_ref(x.double().numpy(), pos, w, mag, 64, False)
    bound = rotate_bound(x.double().numpy(), w, mag, 64, False, True, ref)
    d = x.to(DEV)
    q, k, v = d[:, :6], d[:, 6:8], d[:, 8:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qo, ko = api.rope(q, k, _t(pos), table, q_out=q, k_out=k)
    side.synchronize()
    assert qo is q and ko is k
    assert_within("q", d[:, :8], torch.from_numpy(ref[:, :8]), torch.from_numpy(bound[:, :8]))
    assert torch.equal(d[:, 8:].cpu(), x[:, 8:])
    none, k2 = api.rope(None, x.to(DEV)[:, 6:8], _t(pos), table)
    assert none is None and torch.equal(k2, ko)
    # heads-major storage and an odd offset (no 16-byte alignment): same numbers
    flat = torch.empty(19 * 6 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    odd = flat[1:].view(6, 19, 64).transpose(0, 1)
    odd.copy_(x.to(DEV)[:, :6])
    assert torch.equal(api.rope(odd, None, _t(pos), table)[0], qo)


def test_rope_records_positions_beyond_the_table():
    w, mag, table = _table(32, positions=50)
    x = _rows(6, 4, 2, 32, torch.float32).to(DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = torch.full_like(x, 7.0)
    api.rope(x, None, _t(np.array([0, 50, -1, 49], np.int32)), table, q_out=out, ws=ws)
    assert api.last_device_error(ws) == 5
    assert bool((out[1:3] == 7).all()) and not bool((out[[0, 3]] == 7).any())
    assert api.last_device_error(ws) == 0


@pytest.mark.parametrize("cache,dtype", [("bf16", torch.bfloat16), ("bf16", torch.float32), ("f32", torch.float32),
                                         ("e4m3", torch.bfloat16), ("e4m3", torch.float32)])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 4, 128, 16), (131, 2, 64, 24), (50, 1, 256, 7), (40, 3, 48, 1), (1000, 8, 128, 64)])
def test_write_and_read_back(cache, dtype, tokens, heads, dim, page):
    pages = -(-tokens // page) + 2
    rng = np.random.default_rng(tokens)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    if tokens > 10:
        slots[[3, 9]] = -1
    k, v = _rows(7, tokens, heads, dim, dtype), _rows(8, tokens, heads, dim, dtype) * 50
    if tokens > 20:
        k[11] = 0.0
        v[12, 0, :] = 1e-30
    c = api.kv_cache(pages, page, heads, dim, cache)
    before = c.k.clone()
    assert api.kv_write(c, k.to(DEV), v.to(DEV), _t(slots)) is None
    keep = slots >= 0
    page_i, at = slots[keep] // page, slots[keep] % page
    for x, got, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        rows = got.cpu()[page_i, at]
        if cache == "e4m3":   # the formula in fp32, code for code
            codes, sc = quantise_ref(x.float()[torch.from_numpy(keep)])
            assert torch.equal(rows, codes)
            assert torch.equal(scales.cpu()[page_i, :, at], sc)
        else:
            assert torch.equal(rows, x.to(rows.dtype)[torch.from_numpy(keep)])
    untouched = np.ones(pages * page, bool)
    untouched[slots[keep]] = False
    assert torch.equal(c.k.flatten(0, 1).cpu()[torch.from_numpy(untouched)], before.flatten(0, 1).cpu()[torch.from_numpy(untouched)])
    for out_type in (torch.bfloat16, torch.float32):
        ko, vo = api.kv_read(c, _t(slots), dtype=out_type)
        for got, store, scales in ((ko, c.k, c.k_scale), (vo, c.v, c.v_scale)):
            x = store.cpu()[page_i, at]
            x = x.view(E4M3).float() * scales.cpu()[page_i, :, at][..., None] if cache == "e4m3" else x.float()
            assert torch.equal(got.cpu()[torch.from_numpy(keep)], x.to(out_type))
            assert not bool(got.cpu()[torch.from_numpy(~keep)].any())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cache,dim,rot", [("e4m3", 128, 128), ("e4m3", 64, 32), ("bf16", 128, 128), ("f32", 40, 20), ("e4m3", 96, 16),
                                           ("e4m3", 48, 18)])
def test_write_with_rotation(cache, dim, rot, interleaved):
    """q, k rotated and k, v written in one call equal the rotation's reference: to fp32 rounding,
    the cache's type, or half a step of the row's code grid (2^-4 relative, 2^-10 scales below)."""
    tokens, hq, hk, page = 23, 8, 2, 16
    w, mag, table = _table(rot)
    pos = np.random.default_rng(1).integers(0, 4096, tokens).astype(np.int32)
    dtype = torch.float32 if cache == "f32" else torch.bfloat16
    q, k, v = _rows(9, tokens, hq, dim, dtype), _rows(10, tokens, hk, dim, dtype), _rows(11, tokens, hk, dim, dtype)
    c = api.kv_cache(4, page, hk, dim, cache)
    slots = np.random.default_rng(2).permutation(4 * page)[:tokens].astype(np.int32)
    slots[5] = -1
    qo = api.kv_write(c, k.to(DEV), v.to(DEV), _t(slots), q=q.to(DEV), positions=_t(pos), table=table, interleaved=interleaved)
    ref = rotate_ref(q.double().numpy(), pos, w, mag, rot, interleaved)
    bound = rotate_bound(q.double().numpy(), w, mag, rot, interleaved, dtype == torch.bfloat16, ref)
    assert_within("q", qo, torch.from_numpy(ref), torch.from_numpy(bound))   # also the token without a slot
    ko, vo = api.kv_read(c, _t(slots), dtype=torch.float32)
    keep = torch.from_numpy(slots >= 0)
    ref = rotate_ref(k.double().numpy(), pos, w, mag, rot, interleaved)
    bound = rotate_bound(k.double().numpy(), w, mag, rot, interleaved, cache == "bf16", ref)
    if cache == "e4m3":
        step = np.abs(ref).max(-1, keepdims=True) / 448
        bound = bound + np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * step) * (1 + 2.0 ** -10) + 2.0 ** -21 * np.abs(ref)
    assert_within("k", ko[keep.to(DEV)], torch.from_numpy(ref)[keep], torch.from_numpy(bound)[keep])
    if cache != "e4m3":
        assert torch.equal(vo.cpu()[keep], v.float()[keep])
    else:
        codes, sc = quantise_ref(v.float())
        assert torch.equal(vo.cpu()[keep], (codes.view(E4M3).float() * sc[..., None])[keep])


def test_write_and_read_record_slots_beyond_the_cache():
    c = api.kv_cache(2, 8, 1, 32, "e4m3")
    x = torch.ones((3, 1, 32), device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    api.kv_write(c, x, x, _t(np.array([0, 16, 2 ** 31 - 1], np.int32)), ws=ws)
    assert api.last_device_error(ws) == 5
    assert int((c.k != 0).sum()) == 32
    ko, vo = api.kv_read(c, _t(np.array([0, 16, -7], np.int32)), ws=ws)
    assert api.last_device_error(ws) == 5
    assert bool((ko[0] == 1).all()) and not bool(ko[1:].any()) and not bool(vo[1:].any())


def test_non_finite_rows_keep_their_places():
    """A NaN stays one element of its row; an infinity makes the row's scale infinite, so its
    finite elements, codes of 0, read back as NaN (0 * inf)."""
    c = api.kv_cache(1, 4, 1, 32, "e4m3")
    x = torch.randn((2, 1, 32), generator=torch.Generator().manual_seed(1))
    x[0, 0, 5] = float("nan")
    x[1, 0, 7] = float("inf")
    api.kv_write(c, x.to(DEV), x.to(DEV), _t(np.array([0, 1], np.int32)))
    ko, _ = api.kv_read(c, _t(np.array([0, 1], np.int32)), dtype=torch.float32)
    assert ko[0, 0].isnan().sum() == 1 and bool(ko[0, 0, 5].isnan())
    assert bool(ko[1].isnan().all())


def test_long_cache_offsets_pass_32_bits():
    """Pages whose element offsets lie beyond 2^32: strided pages of one large buffer."""
    page, heads, dim, pages = 16, 1, 128, 5
    stride = (1 << 30) + 4096
    big = torch.empty(stride * (pages - 1) + page * heads * dim, dtype=torch.uint8, device=DEV)
    view = big.as_strided((pages, page, heads, dim), (stride, heads * dim, dim, 1))
    scales = [torch.ones((pages, heads, page), device=DEV) for _ in range(2)]
    bigv = torch.empty_like(big)
    c = api.KVCache(view, bigv.as_strided(view.shape, view.stride()), *scales)
    x = _rows(12, 3, heads, dim, torch.bfloat16).to(DEV)
    slots = _t(np.array([4 * page + 3, 0, 3 * page + 15], np.int32))
    api.kv_write(c, x, -x, slots)
    ko, vo = api.kv_read(c, slots, dtype=torch.float32)
    codes, sc = quantise_ref(x.cpu().float())
    assert torch.equal(ko.cpu(), codes.view(E4M3).float() * sc[..., None]) and torch.equal(vo, -ko)


def test_empty_calls():
    w, mag, table = _table(32)
    e = torch.empty((0, 2, 32), device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert api.rope(e, e, none, table)[0].shape == (0, 2, 32)
    c = api.kv_cache(1, 4, 2, 32, "f32")
    api.kv_write(c, e, e, none)
    assert api.kv_read(c, none)[0].shape == (0, 2, 32)

"""Refusals of the latent cache's and the pages' calls, on the host and before any launch; and that the
binding makes their tensors' device current."""
import contextlib
import ctypes
import struct
import types

import pytest
import torch

from moe_speculative_decoding_gb300 import api
from moe_speculative_decoding_gb300 import build as mbuild

ARG, UNSUPPORTED, WORKSPACE = 1, 2, 4
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return api.lib()


def latent(**kw):
    d = dict(rows=4096, page_stride=64 * 576, token_stride=576, dtype=1, rank=512, rope=64, page=64, pages=8, reserved=0)
    return api.LatentDesc(**{**d, **kw})


def heads(ptr=4096, token_stride=576, head_stride=576, n=1, dtype=1):
    return struct.pack("@Pqqii", ptr, token_stride, head_stride, n, dtype)


def rotary(table=4096, positions=4096, table_positions=100, rot=64):
    return struct.pack("@PPiiii", table, positions, table_positions, rot, 0, 0)


# descriptors that the cache's rules refuse
BAD_CACHES = [(dict(rows=None), ARG), (dict(rows=4104), ARG), (dict(dtype=2), ARG), (dict(reserved=1), ARG), (dict(rank=0), ARG),
              (dict(rope=0), ARG), (dict(page=0), ARG), (dict(pages=0), ARG), (dict(rank=520), UNSUPPORTED), (dict(rope=136), UNSUPPORTED),
              (dict(rank=508), UNSUPPORTED), (dict(rope=4), UNSUPPORTED), (dict(page=1 << 16, pages=1 << 15), UNSUPPORTED),
              (dict(token_stride=577), ARG), (dict(page_stride=-576), ARG)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches(lib, change, code):
    c = ctypes.byref(latent(**change))
    assert lib.moe_latent_write(c, heads(), heads(), 4096, 4, None, 0.0, None, None, None, None, None) == code
    assert lib.moe_latent_attention(c, heads(n=16), heads(n=16), None, 4096, 4096, 4096, None, 1, 4, 4, 4, 1.0, 4096, BIG, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(cache=None), ARG), (dict(tokens=-1), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("inf")), ARG), (dict(eps=float("nan")), ARG),
    (dict(latent=None), ARG), (dict(latent=heads(n=2)), ARG), (dict(k=heads(n=2)), ARG), (dict(k=heads(ptr=0)), ARG),
    (dict(latent=heads(dtype=2)), ARG), (dict(latent=heads(ptr=4097)), ARG), (dict(slots=None), ARG), (dict(slots=4098), ARG),
    (dict(norm=4097), ARG), (dict(ws=4100), ARG), (dict(q=heads(n=4)), ARG), (dict(q=heads(n=4), q_out=heads(n=4)), ARG),
    (dict(q=heads(n=4), q_out=heads(n=5), rot=rotary()), ARG), (dict(rot=rotary(rot=66)), ARG), (dict(rot=rotary(rot=7)), ARG),
    (dict(rot=rotary(table=0)), ARG), (dict(rot=rotary(table=4100)), ARG), (dict(rot=rotary(table_positions=0)), ARG),
    (dict(tokens=1 << 30, q=heads(n=4), q_out=heads(n=4), rot=rotary()), UNSUPPORTED), (dict(tokens=0), 0), (dict(tokens=0, latent=None), 0)])
def test_write(lib, change, code):
    a = dict(cache=ctypes.byref(latent()), latent=heads(), k=heads(), slots=4096, tokens=4, norm=None, eps=1e-6, rot=None, q=None,
             q_out=None, ws=None)
    a.update(change)
    assert lib.moe_latent_write(*a.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(cache=None), ARG), (dict(seqs=-1), ARG), (dict(tokens=-1), ARG), (dict(max_tokens=0), ARG), (dict(max_pages=0), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(max_tokens=65), UNSUPPORTED), (dict(seqs=65536), UNSUPPORTED), (dict(q=None), ARG), (dict(out=heads(n=15)), ARG),
    (dict(out=heads(n=16, dtype=0)), ARG), (dict(q=heads(n=1025), out=heads(n=1025)), UNSUPPORTED), (dict(q_start=None), ARG),
    (dict(ctx=4098), ARG), (dict(pages=None), ARG), (dict(mask=4100), ARG), (dict(lse=4097), ARG), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE), (dict(ws=4104), ARG), (dict(tokens=0), 0), (dict(seqs=0), 0)])
def test_attention(lib, change, code):
    a = dict(cache=ctypes.byref(latent()), q=heads(n=16), out=heads(n=16), lse=None, q_start=4096, ctx=4096, pages=4096, mask=None,
             seqs=1, tokens=4, max_tokens=4, max_pages=4, scale=1.0, ws=4096, ws_bytes=BIG)
    a.update(change)
    assert lib.moe_latent_attention(*a.values(), None) == code


def test_workspaces(lib):
    need = lib.moe_latent_attention_workspace_bytes
    assert need(ctypes.byref(latent()), 64, 4, 16) > need(ctypes.byref(latent(dtype=0)), 64, 4, 16) > 256
    assert need(None, 64, 4, 16) == need(ctypes.byref(latent()), -1, 4, 16) == 0
    assert lib.moe_pages_workspace_bytes(ctypes.byref(pool())) >= 256 + 4 * 100 + 16 * 8
    assert lib.moe_pages_workspace_bytes(None) == lib.moe_pages_workspace_bytes(ctypes.byref(pool(seqs=0))) == 0


def pool(**kw):
    d = dict(refs=4096, table=4096, held=4096, pages=100, page=64, seqs=8, max_pages=10)
    return api.PoolDesc(**{**d, **kw})


def caches(kv=(), lat=(), **kw):
    a, b = (api.CacheDesc * max(1, len(kv)))(*kv), (api.LatentDesc * max(1, len(lat)))(*lat)
    c = api.CachesDesc(ctypes.addressof(a), ctypes.addressof(b), len(kv), len(lat))
    for k, v in kw.items():
        setattr(c, k, v)
    c.keep = (a, b)
    return c


def kv_desc(**kw):
    d = dict(k=4096, v=4096, k_scale=None, v_scale=None, page_stride=64 * 256, token_stride=256, head_stride=128, dtype=1, heads=2,
             dim=128, page=64, pages=100, reserved=0)
    return api.CacheDesc(**{**d, **kw})


BAD_POOLS = [(dict(refs=None), ARG), (dict(table=None), ARG), (dict(held=4097), ARG), (dict(pages=0), ARG), (dict(page=0), ARG),
             (dict(seqs=0), ARG), (dict(max_pages=0), ARG), (dict(max_pages=1 << 26), UNSUPPORTED), (dict(pages=1 << 26), UNSUPPORTED),
             (dict(seqs=1 << 20, max_pages=1 << 12), UNSUPPORTED)]


@pytest.mark.parametrize("change,code", BAD_POOLS)
def test_bad_pools(lib, change, code):
    p, c = ctypes.byref(pool(**change)), ctypes.byref(caches(lat=[latent(pages=100)]))
    assert lib.moe_pages_reserve(p, 4096, 4096, None, c, 4096, BIG, None) == code
    assert lib.moe_pages_fork(p, 4096, 4096, 2, 4096, 4096, BIG, None) == code
    assert lib.moe_pages_accept(p, 4096, 4096, 4096, 4, None, c, 4096, BIG, None) == code
    assert lib.moe_pages_free(p, 4096, 2, None, 4096, BIG, None) == code


@pytest.mark.parametrize("c,code", [
    (None, ARG), (caches(kv=[kv_desc(pages=99)]), ARG), (caches(kv=[kv_desc(page=32)]), ARG), (caches(kv=[kv_desc(k=None)]), ARG),
    (caches(kv=[kv_desc(dtype=2)]), ARG), (caches(lat=[latent(pages=7)]), ARG), (caches(lat=[latent(pages=100, rank=520)]), UNSUPPORTED),
    (caches(kv_count=-1), ARG), (caches(latent_count=-2), ARG),
    # 1025 caches of equal shape are more launches than a call makes
    (caches(lat=[latent(pages=100)] * 1025), UNSUPPORTED)])
def test_bad_lists_of_caches(lib, c, code):
    p, c = ctypes.byref(pool()), None if c is None else ctypes.byref(c)
    assert lib.moe_pages_reserve(p, 4096, 4096, None, c, 4096, BIG, None) == code
    assert lib.moe_pages_accept(p, 4096, 4096, 4096, 4, None, c, 4096, BIG, None) == code


def test_page_calls(lib):
    p, c = ctypes.byref(pool()), ctypes.byref(caches(kv=[kv_desc()]))
    many = ctypes.byref(pool(seqs=1025))
    assert lib.moe_pages_reserve(many, 4096, 4096, None, c, 4096, BIG, None) == UNSUPPORTED
    for args, code in (((None, 4096, None, c, 4096, BIG), ARG), ((4096, None, None, c, 4096, BIG), ARG), ((4096, 4096, 4097, c, 4096, BIG), ARG),
                       ((4096, 4096, None, c, None, BIG), WORKSPACE), ((4096, 4096, None, c, 4096, 256), WORKSPACE),
                       ((4096, 4096, None, c, 4104, BIG), ARG)):
        assert lib.moe_pages_reserve(p, *args, None) == code
    for args, code in (((4096, 4096, -1, 4096, 4096, BIG), ARG), ((4096, 4096, 1025, 4096, 4096, BIG), UNSUPPORTED), ((None, None, 0, None, None, 0), 0),
                       ((None, 4096, 2, 4096, 4096, BIG), ARG), ((4096, 4098, 2, 4096, 4096, BIG), ARG), ((4096, 4096, 2, None, 4096, BIG), ARG),
                       ((4096, 4096, 2, 4096, 4096, 300), WORKSPACE)):
        assert lib.moe_pages_fork(p, *args, None) == code
    for args, code in (((4096, 4096, 4096, 0, None, c, 4096, BIG), ARG), ((4096, 4096, 4096, 65, None, c, 4096, BIG), UNSUPPORTED),
                       ((None, 4096, 4096, 4, None, c, 4096, BIG), ARG), ((4096, 4097, 4096, 4, None, c, 4096, BIG), ARG),
                       ((4096, None, None, 4, None, c, 4096, BIG), ARG), ((4096, 4096, 4096, 4, 4098, c, 4096, BIG), ARG),
                       ((4096, 4096, 4096, 4, None, c, 4096, 400), WORKSPACE)):
        assert lib.moe_pages_accept(p, *args, None) == code
    for args, code in (((4096, -1, None, 4096, BIG), ARG), ((None, 0, None, None, 0), 0), ((None, 3, None, 4096, BIG), ARG),
                       ((4096, 3, 4097, 4096, BIG), ARG), ((4096, 3, None, None, BIG), WORKSPACE)):
        assert lib.moe_pages_free(p, *args, None) == code


# ---------------------------------------------------------------- the binding
class There(torch.Tensor):
    """A tensor of cuda:1, as far as the binding can see."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(There)


def _i32(*shape):
    return _t(*shape, dtype=torch.int32)


@pytest.fixture
def entered(monkeypatch):
    """{call: the device current when it was entered}."""
    seen, current = {}, [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d if isinstance(d, int) else d.index
        try:
            yield
        finally:
            current[0] = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen[name] = current[0]
                return 4096 if name.endswith("_bytes") else 0
            return call

    monkeypatch.setattr(api, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(api, "_current_device", torch.cuda.current_device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)
    empty, zeros = torch.empty, torch.zeros
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k).as_subclass(There))
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k).as_subclass(There))
    yield seen
    assert current[0] == 0


def test_tensors_device_is_current(entered):
    cache = api.LatentCache(_t(4, 8, 40), 32)
    slots, table = _i32(3), _t(9, 4, 2)
    q = api.latent_write(cache, _t(3, 32), _t(3, 8), slots, norm=_t(32), q=_t(3, 2, 8), positions=slots, table=table)
    assert q.shape == (3, 2, 8)
    out, lse = api.latent_attention(cache, _t(3, 2, 40), _i32(2), _i32(1), _i32(1, 2), 1.0, return_lse=True)
    assert out.shape == (3, 2, 32) and lse.shape == (3, 2)
    pool = api.page_pool([cache, api.KVCache(_t(4, 8, 2, 4), _t(4, 8, 2, 4))], 2, 3)
    assert api.pages_reserve(pool, _i32(2), _i32(2)).shape == (2,)
    api.pages_fork(pool, _i32(1), _i32(1), _i32(2))
    assert api.pages_accept(pool, _i32(2), _i32(2, 4), _i32(2)).shape == (2,)
    api.pages_accept(pool, _i32(2), None, _i32(2))
    api.pages_free(pool, _i32(2))
    launching = {k: v for k, v in entered.items() if k != "moe_pages_workspace_bytes"}
    assert set(launching) == {"moe_latent_write", "moe_latent_attention", "moe_latent_attention_workspace_bytes", "moe_workspace_init",
                              "moe_pages_reserve", "moe_pages_fork", "moe_pages_accept", "moe_pages_free"}
    assert set(launching.values()) == {1}, entered


def test_binding_refuses(entered):
    cache, slots, table, w = api.LatentCache(_t(4, 8, 40), 32), _i32(3), _t(9, 4, 2), torch.ones
    with pytest.raises(TypeError):
        api.LatentCache(w(4, 8, 40), 32)                       # on the host
    with pytest.raises(TypeError):
        api.LatentCache(_t(4, 8, 40, dtype=torch.float16), 32)
    for rank in (0, 40, 41):
        with pytest.raises(ValueError):
            api.LatentCache(_t(4, 8, 40), rank)
    with pytest.raises(ValueError):
        api.LatentCache(_t(4, 8, 80)[..., ::2], 32)
    for change in (dict(latent=_t(3, 31)), dict(k_rope=_t(2, 8)), dict(k_rope=_t(3, 16)[:, ::2]), dict(positions=slots), dict(table=table),
                   dict(q=_t(3, 2, 8)), dict(q_out=_t(3, 2, 8)), dict(norm=_t(31)), dict(slots=_i32(2)),
                   dict(q=_t(3, 2, 4), positions=slots, table=table)):
        with pytest.raises(ValueError):
            api.latent_write(**{**dict(cache=cache, latent=_t(3, 32), k_rope=_t(3, 8), slots=slots), **change})
    for change in (dict(latent=w(3, 32)), dict(slots=_t(3)), dict(norm=_t(32, dtype=torch.bfloat16)), dict(ws=w(9))):
        with pytest.raises(TypeError):
            api.latent_write(**{**dict(cache=cache, latent=_t(3, 32), k_rope=_t(3, 8), slots=slots), **change})
    ok = dict(cache=cache, q=_t(3, 2, 40), q_start=_i32(2), ctx=_i32(1), page_table=_i32(1, 2), scale=1.0)
    for change in (dict(q=_t(3, 2, 39)), dict(q_start=_i32(3)), dict(ctx=_i32(2)), dict(out=_t(3, 2, 31)), dict(lse=_t(3, 1)),
                   dict(mask=_t(2, dtype=torch.int64)), dict(page_table=_i32(1, 4)[:, ::2])):
        with pytest.raises(ValueError):
            api.latent_attention(**{**ok, **change})
    for change in (dict(q_start=_t(2)), dict(mask=_i32(3)), dict(q=w(3, 2, 40))):
        with pytest.raises(TypeError):
            api.latent_attention(**{**ok, **change})
    pool = api.page_pool([cache], 2, 3)
    with pytest.raises(ValueError):
        api.PagePool([], _i32(4), _i32(2, 3), _i32(2))
    with pytest.raises(TypeError):
        api.PagePool([_t(4)], _i32(4), _i32(2, 3), _i32(2))
    with pytest.raises(ValueError):
        api.PagePool([cache, api.LatentCache(_t(5, 8, 40), 32)], _i32(4), _i32(2, 3), _i32(2))
    for refs, table, held in ((_i32(5), _i32(2, 3), _i32(2)), (_i32(4), _i32(6), _i32(2)), (_i32(4), _i32(2, 3), _i32(3))):
        with pytest.raises(ValueError):
            api.PagePool([cache], refs, table, held)
    with pytest.raises(ValueError):
        api.pages_reserve(pool, _i32(3), _i32(2))
    with pytest.raises(TypeError):
        api.pages_reserve(pool, _i32(2), _t(2))
    with pytest.raises(ValueError):
        api.pages_fork(pool, _i32(1), _i32(2), _i32(2))
    with pytest.raises(ValueError):
        api.pages_accept(pool, _i32(2), _i32(2), _i32(2))
    with pytest.raises(ValueError):
        api.pages_free(pool, _i32(1), _i32(3))

"""The attention side on the CPU: rotary frequencies against their formulas, and the refusals of
every call (all before any launch: there is no GPU here)."""
import ctypes

import numpy as np
import pytest
import torch

from moe_speculative_decoding_gb300 import api
from moe_speculative_decoding_gb300 import build as mbuild

P = ctypes.c_void_p
BUF = 0x10000   # an aligned address that nothing reads: every check is on the host


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return api.lib()


@pytest.mark.parametrize("rot,base", [(128, 1e6), (64, 1e4), (2, 500.0), (90, 1e4), (256, 1e4)])
def test_frequencies(lib, rot, base):
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    w, m = api.rope_frequencies(rot, base)
    assert np.allclose(w, plain, rtol=1e-13) and m == 1.0
    w, m = api.rope_frequencies(rot, base, "linear", 4.0)
    assert np.allclose(w, plain / 4, rtol=1e-13) and m == 1.0
    w, m = api.rope_frequencies(rot, base, "base", 8.0)
    assert m == 1.0 and w[0] == 1.0
    if rot > 2:   # the slowest is divided by the factor, to the last bit of pow
        assert np.isclose(w[-1], plain[-1] / 8, rtol=1e-12)


def test_frequencies_by_parts(lib):
    rot, base, factor, original = 128, 1e4, 16.0, 4096
    w, m = api.rope_frequencies(rot, base, "by_parts", factor, original, 32.0, 1.0)
    plain = base ** (-2.0 * np.arange(64) / rot)
    turns = original * plain / (2 * np.pi)
    assert np.isclose(m, 0.1 * np.log(16.0) + 1, rtol=1e-14)
    assert np.allclose(w[turns > 40], plain[turns > 40], rtol=1e-13)                # fast ones keep
    assert np.allclose(w[turns < 0.8], plain[turns < 0.8] / factor, rtol=1e-13)     # slow ones are interpolated
    ratio = plain / w
    assert np.all(np.diff(ratio) >= -1e-12) and ratio[0] == 1.0 and np.isclose(ratio[-1], factor)
    lo = np.floor(rot * np.log(original / (2 * np.pi * 32.0)) / (2 * np.log(base)))
    hi = np.ceil(rot * np.log(original / (2 * np.pi)) / (2 * np.log(base)))
    ramp = np.clip((np.arange(64) - lo) / (hi - lo), 0, 1)
    assert np.allclose(w, plain * (ramp / factor + 1 - ramp), rtol=1e-13)


def test_frequency_refusals(lib):
    out = (ctypes.c_double * 128)()
    mag = ctypes.c_double()
    f = lambda rot=64, base=1e4, sc=0, fac=1.0, orig=0, bf=32.0, bs=1.0, w=out: lib.moe_rope_frequencies(
        rot, base, sc, fac, orig, bf, bs, w, ctypes.byref(mag))
    assert f() == 0
    for bad in (dict(rot=0), dict(rot=3), dict(rot=258), dict(base=1.0), dict(base=float("nan")), dict(fac=0.5),
                dict(fac=float("inf")), dict(sc=4), dict(sc=-1), dict(sc=3), dict(sc=3, orig=100, bs=0.0),
                dict(sc=3, orig=100, bs=32.0), dict(w=None)):
        assert f(**bad) == 1, bad
    assert lib.moe_rope_table(out, 0, 1.0, 4, BUF, None) == 1
    assert lib.moe_rope_table(out, 129, 1.0, 4, BUF, None) == 1
    assert lib.moe_rope_table(out, 4, 1.0, -1, BUF, None) == 1
    assert lib.moe_rope_table(out, 4, 1.0, 4, BUF + 4, None) == 1
    assert lib.moe_rope_table(out, 4, 1.0, 0, None, None) == 0


def _cache(**over):
    f = dict(k=BUF, v=BUF, k_scale=None, v_scale=None, page_stride=16 * 2 * 64, token_stride=128, head_stride=64,
             dtype=1, heads=2, dim=64, page=16, pages=8, reserved=0)
    f.update(over)
    return api.CacheDesc(*[f[n] for n, _ in api.CacheDesc._fields_])


def _heads(**over):
    f = dict(ptr=BUF, token_stride=128, head_stride=64, heads=2, dtype=1)
    f.update(over)
    return api.Heads(*[f[n] for n, _ in api.Heads._fields_])


def _rot(**over):
    f = dict(table=BUF, positions=BUF, table_positions=100, rot=64, interleaved=0, inverse=0)
    f.update(over)
    return api.Rotary(*[f[n] for n, _ in api.Rotary._fields_])


def _ref(x):
    return None if x is None else ctypes.byref(x)


def test_rope_refusals(lib):
    def call(q=_heads(), qo=_heads(), k=None, ko=None, tokens=4, dim=64, rot=_rot(), ws=None):
        return lib.moe_rope(_ref(q), _ref(qo), _ref(k), _ref(ko), tokens, dim, _ref(rot), ws, None)
    assert call(tokens=0) == 0
    for bad in (dict(tokens=-1), dict(dim=0), dict(rot=None), dict(rot=_rot(rot=66)), dict(rot=_rot(rot=3)), dict(rot=_rot(rot=0)),
                dict(rot=_rot(table=BUF + 4)), dict(rot=_rot(positions=None)), dict(rot=_rot(table_positions=0)),
                dict(q=None), dict(qo=None), dict(q=None, qo=None), dict(k=_heads()), dict(q=_heads(ptr=None)),
                dict(q=_heads(ptr=BUF + 1)), dict(q=_heads(dtype=2)), dict(q=_heads(heads=0)), dict(qo=_heads(heads=3)),
                dict(ws=BUF + 8)):
        assert call(**bad) == 1, bad
    assert call(dim=257) == 2
    assert call(tokens=1 << 30, q=_heads(heads=4), qo=_heads(heads=4)) == 2   # 2^32 rows


def test_cache_refusals(lib):
    def write(c=_cache(), k=_heads(), v=_heads(), slots=BUF, tokens=4, rot=None, q=None, qo=None, ws=None):
        return lib.moe_kv_write(_ref(c), _ref(k), _ref(v), slots, tokens, _ref(rot), _ref(q), _ref(qo), ws, None)

    def read(c=_cache(), k=_heads(), v=_heads(), slots=BUF, tokens=4, ws=None):
        return lib.moe_kv_read(_ref(c), slots, tokens, _ref(k), _ref(v), ws, None)

    bad_caches = [(None, 1), (_cache(reserved=1), 1), (_cache(dtype=3), 1), (_cache(heads=0), 1), (_cache(dim=0), 1),
                  (_cache(page=0), 1), (_cache(pages=0), 1), (_cache(dim=264), 2), (_cache(dim=60), 2), (_cache(k=None), 1),
                  (_cache(v=BUF + 8), 1), (_cache(token_stride=100), 1), (_cache(page_stride=-128), 1), (_cache(dtype=2), 1),
                  (_cache(dtype=2, k_scale=BUF, v_scale=BUF + 2), 1), (_cache(pages=1 << 28), 2)]
    for c, status in bad_caches:
        assert write(c=c) == status and read(c=c) == status
    assert write(tokens=0) == 0 and read(tokens=0) == 0
    for f in (write, read):
        for bad in (dict(tokens=-1), dict(k=None), dict(v=None), dict(k=_heads(heads=1)), dict(v=_heads(dtype=2)), dict(slots=None),
                    dict(slots=BUF + 2), dict(ws=BUF + 4)):
            assert f(**bad) == 1, bad
        assert f(tokens=1 << 30) == 2
    for bad in (dict(q=_heads(), qo=_heads()), dict(rot=_rot(), q=_heads()), dict(rot=_rot(), qo=_heads()), dict(rot=_rot(rot=128)),
                dict(rot=_rot(), q=_heads(), qo=_heads(heads=4))):
        assert write(**bad) == 1, bad


def test_tree_attention_refusals(lib):
    def call(c=_cache(), q=_heads(heads=4), out=_heads(heads=4), lse=None, qs=BUF, ctx=BUF, pt=BUF, mask=None, seqs=2, tokens=8,
             mt=8, mp=4, scale=0.125, ws=BUF, nbytes=1 << 40):
        return lib.moe_tree_attention(_ref(c), _ref(q), _ref(out), lse, qs, ctx, pt, mask, seqs, tokens, mt, mp, scale, ws, nbytes, None)
    assert call(tokens=0) == 0 and call(seqs=0) == 0
    for bad in (dict(c=None), dict(seqs=-1), dict(tokens=-1), dict(mt=0), dict(mp=0), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=None), dict(out=None), dict(out=_heads(heads=2)), dict(out=_heads(heads=4, dtype=0)),
                dict(q=_heads(heads=3), out=_heads(heads=3)), dict(qs=None), dict(ctx=None), dict(pt=None), dict(mask=BUF + 4),
                dict(lse=BUF + 2), dict(ws=BUF + 8)):
        assert call(**bad) == 1, bad
    assert call(mt=65) == 2 and call(seqs=65536) == 2
    assert call(q=_heads(heads=130), out=_heads(heads=130)) == 2   # 65 query heads to a cache head
    assert call(ws=None) == 4
    need = lib.moe_tree_attention_workspace_bytes(ctypes.byref(_cache()), 8, 2, 4)
    assert need >= 256 and call(nbytes=need - 1) == 4
    assert lib.moe_tree_attention_workspace_bytes(None, 8, 2, 4) == 0


def test_binding_refusals():
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        api.KVCache(torch.zeros((2, 4, 1, 64)), torch.zeros((2, 4, 1, 64)))
    with pytest.raises(TypeError):
        api._heads(x, "q", 2, 2, 64, 0)

"""A call's kernels go to the device that is current when the library is entered, so the binding makes
it the tensors' own.  Shown with tensors that say they are on a second device and a library that
notes which device is current: nothing is launched."""
import contextlib
import types

import pytest
import torch

from moe_speculative_decoding_gb300 import api


class There(torch.Tensor):
    """A tensor of cuda:1, as far as the binding can see."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(There)


@pytest.fixture
def entered(monkeypatch):
    """{call: the device current when it was entered}."""
    seen, current = {}, [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d if isinstance(d, int) else d.index
        yield
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
    plain = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: plain(*a, **k).as_subclass(There))
    yield seen
    assert current[0] == 0


def _i32(*shape):
    return _t(*shape, dtype=torch.int32)


def test_attention_side(entered):
    table, positions, rows = api.rope_table(9, [1.0, 0.5]), _i32(3), _t(3, 2, 4)
    api.rope(rows, rows, positions, table)
    cache = api.KVCache(_t(2, 8, 2, 4), _t(2, 8, 2, 4))
    api.kv_write(cache, rows, rows, positions, q=rows, positions=positions, table=table)
    api.kv_read(cache, positions, dtype=torch.float32)
    api.tree_attention(cache, rows, _i32(2), _i32(1), _i32(1, 2))
    assert set(entered) >= {"moe_rope_table", "moe_rope", "moe_kv_write", "moe_kv_read", "moe_tree_attention",
                            "moe_tree_attention_workspace_bytes", "moe_workspace_init"}
    assert set(entered.values()) == {1}, entered


def test_expert_side(entered):
    layer = api.make_layer(16, 8, 4, 2, "f32")
    weights = (_t(4, 8, 16), _t(4, 8, 16), _t(4, 16, 8))
    x, ids, gates, ws = _t(3, 16), _i32(3, 2), _t(3, 2), api.workspace(layer)
    api.route_topm(_t(3, 4), 2)
    grouping = api.Grouping(_i32(1), _i32(4), _i32(5), _i32(6))
    api.group_slots(ids, 4, out=grouping, ws=ws)
    api.expert_op_perslot(layer, weights, x, ids, gates, ws=ws)
    api.expert_op_dedup_ids(layer, weights, x, ids, gates, ws=ws)
    api.expert_op_dedup(layer, weights, x, gates, grouping, ws=ws)
    api.quantize_rows_e4m3(x)
    codes, u8 = api.make_layer(16, 8, 4, 2, "e4m3"), lambda *s: _t(*s, dtype=torch.uint8)
    weights, scales = (u8(4, 8, 16), u8(4, 8, 16), u8(4, 16, 8)), (_t(4, 8), _t(4, 8), _t(4, 16))
    api.expert_op_perslot_fp8(codes, weights, scales, u8(3, 16), _t(3), ids, gates, ws=ws)
    api.expert_op_dedup_ids_fp8(codes, weights, scales, u8(3, 16), _t(3), ids, gates, ws=ws)
    api.expert_op_dedup_fp8(codes, weights, scales, u8(3, 16), _t(3), gates, grouping, ws=ws)
    api.spec_accept(_i32(2, 1), _t(2, 1, 5), _t(2, 2, 5), _t(2, 1), _t(2))
    api.union_cost(_t(3, 1, 1, dtype=torch.int64), _i32(4), _t(2, dtype=torch.float64), _t(3, dtype=torch.float64), 1.0)
    api.read_probe(_t(64), ws)
    api.last_device_error(ws)
    launching = {k: v for k, v in entered.items() if not k.endswith("_bytes")}
    assert len(launching) == 14 and set(launching.values()) == {1}, entered


def test_host_tensors_are_still_refused():
    layer, w = api.make_layer(16, 8, 4, 2, "f32"), torch.zeros
    with pytest.raises(TypeError):
        api.route_topm(w(3, 4), 2)
    with pytest.raises(TypeError):
        api.quantize_rows_e4m3(w(3, 16))
    with pytest.raises(TypeError):
        api.expert_op_dedup_ids(layer, (w(4, 8, 16), w(4, 8, 16), w(4, 16, 8)), w(3, 16), w(3, 2), w(3, 2), ws=w(9))
    with pytest.raises(TypeError):
        api.rope(w(3, 2, 4), None, w(3), w(4, 2, 2))

"""Python binding of libmoeverify.so: argument marshalling only.

Every step of the verify-pass expert operation runs in the library's CUDA kernels; this
module checks tensor devices, dtypes and shapes, passes raw pointers and the current
torch stream, and turns status codes into exceptions.  There is no fallback: if the
library is missing, every call raises MoeError.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import numpy as np
import torch

from . import build as _build

MOE_F32, MOE_BF16, MOE_E4M3 = 0, 1, 2
MOE_FLAG_SIMT = 1
MAX_PASS_TOKENS = 64        # tokens per pass of every expert-operation call
PERSLOT_LAUNCH_TOKENS = 16  # tokens per launch of the per-slot calls (a longer pass is split)
MAX_PERSLOT_TOKENS = 64     # tokens per per-slot call
STATUS = {0: "MOE_OK", 1: "MOE_ERR_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CUDA",
          4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_BAD_ID", 6: "MOE_ERR_DEVICE_TIMEOUT"}


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


class Layer(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("f", ctypes.c_int32), ("N", ctypes.c_int32),
                ("m", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]

    @property
    def torch_dtype(self):
        if self.w_dtype == MOE_E4M3:
            return torch.uint8   # e4m3 codes
        return torch.bfloat16 if self.w_dtype == MOE_BF16 else torch.float32


class _PassBytes(ctypes.Structure):
    _fields_ = [("expert_bytes", ctypes.c_uint64), ("slot_bytes", ctypes.c_uint64),
                ("dedup_bytes", ctypes.c_uint64), ("act_bytes", ctypes.c_uint64),
                ("n", ctypes.c_int32), ("m", ctypes.c_int32), ("U", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("ubar", ctypes.c_double)]


class WeightScales(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class Heads(ctypes.Structure):
    """moe_heads_t: [tokens, heads, dim] rows (element strides)."""
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class CacheDesc(ctypes.Structure):
    """moe_kv_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)] + \
               [(f, ctypes.c_int32) for f in ("dtype", "heads", "dim", "page", "pages", "reserved")]


class Rotary(ctypes.Structure):
    """moe_rotary_t."""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p)] + \
               [(f, ctypes.c_int32) for f in ("table_positions", "rot", "interleaved", "inverse")]


class LatentDesc(ctypes.Structure):
    """moe_latent_cache_t."""
    _fields_ = [("rows", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)] + \
               [(f, ctypes.c_int32) for f in ("dtype", "rank", "rope", "page", "pages", "reserved")]


class PoolDesc(ctypes.Structure):
    """moe_page_pool_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("refs", "table", "held")] + \
               [(f, ctypes.c_int32) for f in ("pages", "page", "seqs", "max_pages")]


class CachesDesc(ctypes.Structure):
    """moe_page_caches_t."""
    _fields_ = [("kv", ctypes.c_void_p), ("latent", ctypes.c_void_p), ("kv_count", ctypes.c_int32),
                ("latent_count", ctypes.c_int32)]


class ThresholdIn(ctypes.Structure):
    _fields_ = [(f, ctypes.c_double) for f in ("mW", "B_k", "beta_1", "tau_1", "dD_over_betaD", "dphi")]


class _ErrorBounds(ctypes.Structure):
    _fields_ = [(f, ctypes.c_double) for f in ("delta", "verify_factor", "decision_log_margin", "regret_factor",
                                               "speedup_lo", "speedup_hi")]


EXPORTED = ("moe_abi_version", "moe_status_str", "moe_workspace_bytes", "moe_workspace_init",
            "moe_route_topm", "moe_group_slots", "moe_expert_op_perslot", "moe_expert_op_dedup",
            "moe_pass_bytes", "moe_bandwidth_report", "moe_expected_union",
            "moe_best_draft_length", "moe_last_device_error", "moe_expert_op_perslot_noalloc",
            "moe_staircase", "moe_speedup", "moe_reuse_threshold", "moe_reuse_threshold_bytes",
            "moe_error_bounds", "moe_kstar_separated", "moe_fit_op_times", "moe_expert_op_perslot_fp8",
            "moe_expert_op_dedup_fp8", "moe_quantize_rows_e4m3", "moe_spec_accept",
            "moe_union_cost_workspace_bytes", "moe_union_cost", "moe_expert_op_dedup_ids",
            "moe_expert_op_dedup_ids_fp8", "moe_read_probe", "moe_set_wait_limit", "moe_rope_frequencies",
            "moe_rope_table", "moe_rope", "moe_kv_write", "moe_kv_read", "moe_tree_attention_workspace_bytes",
            "moe_tree_attention", "moe_latent_write", "moe_latent_attention_workspace_bytes", "moe_latent_attention",
            "moe_pages_workspace_bytes", "moe_pages_reserve", "moe_pages_fork", "moe_pages_accept", "moe_pages_free")

_lib = None


def lib_path() -> str:
    """Path of the in-tree libmoeverify.so (library infrastructure)."""
    return _build.LIB


def lib():
    """The loaded library.  Raises MoeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise MoeError(-1, f"libmoeverify.so not built at {path} "
                           "(run python -m moe_speculative_decoding_gb300.build)")
    L = ctypes.CDLL(path)
    P, I32, SZ, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_double
    LP = ctypes.POINTER(Layer)
    sig = {
        "moe_abi_version": ([], I32),
        "moe_status_str": ([I32], ctypes.c_char_p),
        "moe_workspace_bytes": ([LP, I32], SZ),
        "moe_workspace_init": ([P, SZ, P], I32),
        "moe_route_topm": ([P, I32, I32, I32, I32, P, P, P], I32),
        "moe_group_slots": ([P, I32, I32, I32, P, P, P, P, P, P], I32),
        "moe_expert_op_perslot": ([LP, P, P, P, P, P, P, I32, I32, P, P, SZ, P], I32),
        "moe_expert_op_dedup": ([LP, P, P, P, P, P, I32, P, P, P, P, I32, P, P, SZ, P], I32),
        "moe_pass_bytes": ([LP, P, I32, ctypes.POINTER(_PassBytes)], I32),
        "moe_bandwidth_report": ([I32, I32, P, P, P, P, P, P, P, P, P, P], I32),
        "moe_expected_union": ([I32, I32, I32], D),
        "moe_best_draft_length": ([P, I32, D], I32),
        "moe_last_device_error": ([P, P, P], I32),
        "moe_set_wait_limit": ([ctypes.c_int64], I32),
        "moe_staircase": ([P, I32, P, P, P, P], I32),
        "moe_speedup": ([P, I32, I32, D], D),
        "moe_reuse_threshold": ([I32, D, ctypes.POINTER(ThresholdIn)], D),
        "moe_reuse_threshold_bytes": ([I32, D, D, D, D], D),
        "moe_error_bounds": ([D, ctypes.POINTER(_ErrorBounds)], I32),
        "moe_kstar_separated": ([P, I32, D, D], I32),
        "moe_fit_op_times": ([I32, P, P, P, I32, D, I32, P], I32),
        "moe_expert_op_perslot_fp8": ([LP, P, P, P, ctypes.POINTER(WeightScales), P, P, P, P, I32, I32, P, P, SZ, P],
                                      I32),
        "moe_expert_op_dedup_fp8": ([LP, P, P, P, ctypes.POINTER(WeightScales), P, P, P, I32, P, P, P, P, I32, P,
                                     P, SZ, P], I32),
        "moe_quantize_rows_e4m3": ([P, I32, I32, I32, P, P, P], I32),
        "moe_spec_accept": ([P, P, P, P, P, I32, I32, I32, I32, P, P, P], I32),
        "moe_expert_op_dedup_ids": ([LP, P, P, P, P, P, P, I32, I32, P, P, SZ, P], I32),
        "moe_expert_op_dedup_ids_fp8": ([LP, P, P, P, ctypes.POINTER(WeightScales), P, P, P, P, I32, I32, P, P, SZ, P],
                                        I32),
        "moe_union_cost_workspace_bytes": ([I32], SZ),
        "moe_read_probe": ([P, SZ, P, P], I32),
        "moe_union_cost": ([P, I32, I32, I32, P, I32, P, P, D, P, P, P, P, P, P, SZ, P], I32),
        "moe_rope_frequencies": ([I32, D, I32, D, I32, D, D, P, P], I32),
        "moe_rope_table": ([P, I32, D, I32, P, P], I32),
        # descriptors go as plain addresses (byref): one conversion less per argument
        "moe_rope": ([P, P, P, P, I32, I32, P, P, P], I32),
        "moe_kv_write": ([P, P, P, P, I32, P, P, P, P, P], I32),
        "moe_kv_read": ([P, P, I32, P, P, P, P], I32),
        "moe_tree_attention_workspace_bytes": ([P, I32, I32, I32], SZ),
        "moe_tree_attention": ([P, P, P, P, P, P, P, P, I32, I32, I32, I32, ctypes.c_float, P, SZ, P], I32),
        "moe_latent_write": ([P, P, P, P, I32, P, ctypes.c_float, P, P, P, P, P], I32),
        "moe_latent_attention_workspace_bytes": ([P, I32, I32, I32], SZ),
        "moe_latent_attention": ([P, P, P, P, P, P, P, P, I32, I32, I32, I32, ctypes.c_float, P, SZ, P], I32),
        "moe_pages_workspace_bytes": ([P], SZ),
        "moe_pages_reserve": ([P, P, P, P, P, P, SZ, P], I32),
        "moe_pages_fork": ([P, P, P, I32, P, P, SZ, P], I32),
        "moe_pages_accept": ([P, P, P, P, I32, P, P, P, SZ, P], I32),
        "moe_pages_free": ([P, P, I32, P, P, SZ, P], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(code: int, what: str):
    if code != 0:
        raise MoeError(code, what)


# Kernels, and the number of SMs they are sized by, go by the current device and not by the tensors':
# every call is made with its tensors' device current.  (torch.cuda.current_device and its checks take
# 2 us of a call that takes 10.)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _there(t: torch.Tensor, fn, *args):
    """fn with t's device current (a call tests for it in line: another function's call would cost it a microsecond)."""
    with torch.cuda.device(t.get_device()):
        return fn(*args)


def _call(name: str, device, *args):
    """A call of the library with a tensor's device current."""
    if device.index == _current_device():
        code = getattr(_lib or lib(), name)(*args)
    else:
        with torch.cuda.device(device.index):
            code = getattr(_lib or lib(), name)(*args)
    if code:
        raise MoeError(code, name)


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------- layer + workspace

def make_layer(d: int, f: int, N: int, m: int, dtype: str = "bf16", simt: bool = False) -> Layer:
    """A moe_layer_t: hidden size d, expert size f, N experts, top-m, weight/activation dtype ([Lan] §1: the expert operation's shapes)."""
    code = {"bf16": MOE_BF16, "f32": MOE_F32, "e4m3": MOE_E4M3}[dtype]
    return Layer(d, f, N, m, code, code, MOE_FLAG_SIMT if simt else 0)


def workspace(layer: Layer, n_max: int = PERSLOT_LAUNCH_TOKENS, device=None) -> torch.Tensor:
    """A zeroed device workspace for passes of up to n_max tokens (moe_workspace_bytes, moe_workspace_init; infrastructure).

    The default serves per-slot calls of any size (they launch 16 tokens at a time); a
    deduplicating call of n > 16 tokens needs n_max >= n."""
    nbytes = int(lib().moe_workspace_bytes(ctypes.byref(layer), n_max))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    _call("moe_workspace_init", ws.device, ctypes.c_void_p(ws.data_ptr()), nbytes, _stream(ws.device))
    return ws


def last_device_error(ws: torch.Tensor) -> int:
    """moe_last_device_error: synchronise, return and clear the workspace's device error code (infrastructure)."""
    code = ctypes.c_int32(0)
    _call("moe_last_device_error", ws.device, ctypes.c_void_p(ws.data_ptr()), _stream(ws.device),
          ctypes.byref(code))
    return int(code.value)


def set_wait_limit(cycles: int) -> None:
    """moe_set_wait_limit: SM cycles one device pipeline wait of later expert and attention calls may take
    before the call records MOE_ERR_DEVICE_TIMEOUT and returns (0: the default; infrastructure)."""
    _check(lib().moe_set_wait_limit(int(cycles)), "moe_set_wait_limit")


# ---------------------------------------------------------------- the hot path

def route_topm(logits: torch.Tensor, m: int, renorm: bool = True, ids=None, gates=None):
    """Top-m routing of fp32 logits [n, N] -> (ids int32 [n, m], gates fp32 [n, m])."""
    if (index := logits.get_device()) >= 0 and index != _current_device():
        return _there(logits, route_topm, logits, m, renorm, ids, gates)
    n, N = logits.shape
    if ids is None:
        ids = torch.empty((n, m), dtype=torch.int32, device=logits.device)
    if gates is None:
        gates = torch.empty((n, m), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route_topm(_dev(logits, "logits", torch.float32), n, N, m, int(bool(renorm)),
                                _dev(ids, "ids", torch.int32, (n, m)),
                                _dev(gates, "gates", torch.float32, (n, m)), _stream(logits.device)),
           "moe_route_topm")
    return ids, gates


@dataclass
class Grouping:
    num_distinct: torch.Tensor   # int32 [1]
    expert_list: torch.Tensor    # int32 [min(N, n*m)]
    offsets: torch.Tensor        # int32 [min(N, n*m) + 1]
    slot_order: torch.Tensor     # int32 [n*m]

    @staticmethod
    def empty(n: int, m: int, N: int, device) -> "Grouping":
        cap = min(N, n * m)
        z = lambda k: torch.zeros(k, dtype=torch.int32, device=device)
        return Grouping(z(1), z(max(cap, 1)), z(cap + 1), z(n * m))


def group_slots(ids: torch.Tensor, N: int, out: Grouping | None = None, ws=None) -> Grouping:
    """moe_group_slots: the pass's slots grouped by expert, a counting sort ([Lan] §1, App. E): U, expert list, offsets, slot order."""
    if (index := ids.get_device()) >= 0 and index != _current_device():
        return _there(ids, group_slots, ids, N, out, ws)
    n, m = ids.shape
    g = out or Grouping.empty(n, m, N, ids.device)
    _check(lib().moe_group_slots(_dev(ids, "ids", torch.int32), n, m, N,
                                 _dev(g.num_distinct, "num_distinct"), _dev(g.expert_list, "expert_list"),
                                 _dev(g.offsets, "offsets"), _dev(g.slot_order, "slot_order"),
                                 ctypes.c_void_p(ws.data_ptr()) if ws is not None else None,
                                 _stream(ids.device)), "moe_group_slots")
    return g


def _weights(layer: Layer, weights):
    wg, wu, wd = weights
    dt = layer.torch_dtype
    return (_dev(wg, "w_gate", dt, (layer.N, layer.f, layer.d)),
            _dev(wu, "w_up", dt, (layer.N, layer.f, layer.d)),
            _dev(wd, "w_down", dt, (layer.N, layer.d, layer.f)))


def _y(layer, x, y):
    n = x.shape[0]
    if y is None:
        y = torch.empty((n, layer.d), dtype=torch.float32, device=x.device)
    return y, _dev(y, "y", torch.float32, (n, layer.d))


def expert_op_perslot(layer: Layer, weights, x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor,
                      y=None, accumulate: bool = False, ws=None):
    """moe_expert_op_perslot: the per-slot form of the expert operation, one expert read per slot ([Lan] §1)."""
    if (index := x.get_device()) >= 0 and index != _current_device():
        return _there(x, expert_op_perslot, layer, weights, x, ids, gates, y, accumulate, ws)
    n = x.shape[0]
    ws = ws if ws is not None else workspace(layer, n, x.device)
    y, yp = _y(layer, x, y)
    _check(lib().moe_expert_op_perslot(ctypes.byref(layer), *_weights(layer, weights),
                                       _dev(x, "x", layer.torch_dtype, (n, layer.d)),
                                       _dev(ids, "ids", torch.int32, (n, layer.m)),
                                       _dev(gates, "gates", torch.float32, (n, layer.m)), n,
                                       int(bool(accumulate)), yp, ctypes.c_void_p(ws.data_ptr()),
                                       ws.numel(), _stream(x.device)), "moe_expert_op_perslot")
    return y


def expert_op_dedup_ids(layer: Layer, weights, x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor,
                        y=None, accumulate: bool = False, ws=None):
    """The deduplicating form from ids in one launch (the grouping built inside the kernel)."""
    if (index := x.get_device()) >= 0 and index != _current_device():
        return _there(x, expert_op_dedup_ids, layer, weights, x, ids, gates, y, accumulate, ws)
    n = x.shape[0]
    ws = ws if ws is not None else workspace(layer, n, x.device)
    y, yp = _y(layer, x, y)
    _check(lib().moe_expert_op_dedup_ids(ctypes.byref(layer), *_weights(layer, weights),
                                         _dev(x, "x", layer.torch_dtype, (n, layer.d)),
                                         _dev(ids, "ids", torch.int32, (n, layer.m)),
                                         _dev(gates, "gates", torch.float32, (n, layer.m)), n,
                                         int(bool(accumulate)), yp, ctypes.c_void_p(ws.data_ptr()),
                                         ws.numel(), _stream(x.device)), "moe_expert_op_dedup_ids")
    return y


def expert_op_dedup(layer: Layer, weights, x: torch.Tensor, gates: torch.Tensor, grouping: Grouping,
                    y=None, accumulate: bool = False, ws=None):
    """moe_expert_op_dedup: the deduplicating form on a precomputed grouping, each distinct expert read once ([Lan] §1)."""
    if (index := x.get_device()) >= 0 and index != _current_device():
        return _there(x, expert_op_dedup, layer, weights, x, gates, grouping, y, accumulate, ws)
    n = x.shape[0]
    ws = ws if ws is not None else workspace(layer, n, x.device)
    y, yp = _y(layer, x, y)
    _check(lib().moe_expert_op_dedup(ctypes.byref(layer), *_weights(layer, weights),
                                     _dev(x, "x", layer.torch_dtype, (n, layer.d)),
                                     _dev(gates, "gates", torch.float32, (n, layer.m)), n,
                                     _dev(grouping.num_distinct, "num_distinct"),
                                     _dev(grouping.expert_list, "expert_list"),
                                     _dev(grouping.offsets, "offsets"),
                                     _dev(grouping.slot_order, "slot_order"),
                                     int(bool(accumulate)), yp, ctypes.c_void_p(ws.data_ptr()),
                                     ws.numel(), _stream(x.device)), "moe_expert_op_dedup")
    return y


# ---------------------------------------------------------------- host-side report

def pass_bytes(layer: Layer, ids_host) -> dict:
    """moe_pass_bytes: E_slot = n m w, E_dedup = U w and u-bar of one pass, on the host ([Lan] §1 "Bytes", §2 "Effective bandwidth")."""
    ids = np.ascontiguousarray(np.asarray(ids_host, dtype=np.int32))
    n = ids.shape[0] if ids.ndim == 2 else ids.size // layer.m
    out = _PassBytes()
    _check(lib().moe_pass_bytes(ctypes.byref(layer), ctypes.c_void_p(ids.ctypes.data), n,
                                ctypes.byref(out)), "moe_pass_bytes")
    return dict(expert_bytes=out.expert_bytes, slot_bytes=out.slot_bytes, dedup_bytes=out.dedup_bytes,
                act_bytes=out.act_bytes, n=out.n, m=out.m, U=out.U, ubar=out.ubar)


def bandwidth_report(n_lo: int, slot_bytes, dedup_bytes, t_slot, t_dedup) -> dict:
    """moe_bandwidth_report: u-bar(n), beta_p, r(n), S(n) and the crossover from bytes and times ([Lan] §2 "Effective bandwidth", §3.1, §2 "Testing the inputs")."""
    arrs = [np.ascontiguousarray(np.asarray(a, dtype=np.float64)) for a in
            (slot_bytes, dedup_bytes, t_slot, t_dedup)]
    count = arrs[0].size
    outs = [np.zeros(count, np.float64) for _ in range(5)]
    cross = ctypes.c_int32(0)
    _check(lib().moe_bandwidth_report(n_lo, count, *[ctypes.c_void_p(a.ctypes.data) for a in arrs],
                                      *[ctypes.c_void_p(o.ctypes.data) for o in outs],
                                      ctypes.byref(cross)), "moe_bandwidth_report")
    res = dict(zip(("beta_slot", "beta_dedup", "ubar", "r", "saving"), outs))
    res["crossover"] = None if cross.value < 0 else int(cross.value)
    return res


def expected_union(N: int, m: int, n: int) -> float:
    """moe_expected_union: E[U] = N (1 - q^n) under uniform routing ([Lan] §1)."""
    return float(lib().moe_expected_union(N, m, n))


def best_draft_length(V, a: float) -> int:
    """moe_best_draft_length: the smallest maximiser k* of G_a(k) / V(k) ([Lan] §1 "Speculative decoding")."""
    V = np.ascontiguousarray(np.asarray(V, dtype=np.float64))
    k = int(lib().moe_best_draft_length(ctypes.c_void_p(V.ctypes.data), V.size - 1, float(a)))
    if k < 0:
        raise MoeError(1, "moe_best_draft_length")
    return k


# ---------------------------------------------------------------- step-time theory
def _times(V) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(V, dtype=np.float64))


def staircase(V) -> dict:
    """a0, the step points a_step[0..kmax] (a_step[0] = 0), alpha[k, i] and the convex flag."""
    V = _times(V)
    K = V.size
    a0 = ctypes.c_double(0.0)
    steps = np.zeros(K, np.float64)
    alpha = np.zeros((K, K), np.float64)
    convex = ctypes.c_int32(0)
    _check(lib().moe_staircase(ctypes.c_void_p(V.ctypes.data), K - 1, ctypes.byref(a0),
                               ctypes.c_void_p(steps.ctypes.data), ctypes.c_void_p(alpha.ctypes.data),
                               ctypes.byref(convex)), "moe_staircase")
    return dict(a0=a0.value, a_step=steps, alpha=alpha, convex=bool(convex.value))


def speedup(V, k: int, a: float) -> float:
    """moe_speedup: T_a(k) / T_a(0) = G_a(k) V(0) / V(k), the speed-up of draft length k ([Lan] §3.2 (9))."""
    V = _times(V)
    return float(lib().moe_speedup(ctypes.c_void_p(V.ctypes.data), V.size - 1, int(k), float(a)))


def reuse_threshold(k: int, a: float, mW: float, B_k: float, beta_1: float, tau_1: float,
                    dD_over_betaD: float = 0.0, dphi: float = 0.0) -> float:
    """moe_reuse_threshold: the deduplicating engine's reuse threshold rho*_k(a) in time ([Lan] §3.4 (14), App. B.2 (B.12)-(B.14))."""
    t = ThresholdIn(mW, B_k, beta_1, tau_1, dD_over_betaD, dphi)
    return float(lib().moe_reuse_threshold(int(k), float(a), ctypes.byref(t)))


def reuse_threshold_bytes(k: int, a: float, mW: float, D_1: float = 0.0, D_k1: float = 0.0) -> float:
    """moe_reuse_threshold_bytes: the same threshold with one bandwidth and no fixed time ([Lan] §3.4 (16), (B.16))."""
    return float(lib().moe_reuse_threshold_bytes(int(k), float(a), float(mW), float(D_1), float(D_k1)))


def error_bounds(eps: float) -> dict:
    """moe_error_bounds: delta, the verify factor of (17)-(18) and the decision margin for a relative bandwidth error eps ([Lan] §3.5, Table 2, App. C)."""
    out = _ErrorBounds()
    _check(lib().moe_error_bounds(float(eps), ctypes.byref(out)), "moe_error_bounds")
    return {f: getattr(out, f) for f, _ in _ErrorBounds._fields_}


def kstar_separated(V, a: float, delta: float) -> bool:
    """moe_kstar_separated: the separation condition of (20), under which the predicted k* is the true one ([Lan] §3.5, Table 2)."""
    V = _times(V)
    r = int(lib().moe_kstar_separated(ctypes.c_void_p(V.ctypes.data), V.size - 1, float(a), float(delta)))
    if r < 0:
        raise MoeError(1, "moe_kstar_separated")
    return bool(r)


def fit_op_times(n, U, t, m: int, b: float, form: str) -> tuple:
    """Fit (4) (form 'slot': t_op, c_u, c_re) or (E.1) (form 'dedup': t_op, c_g, c_t)."""
    n = np.ascontiguousarray(np.asarray(n, dtype=np.int32))
    U = np.ascontiguousarray(np.asarray(U, dtype=np.int32))
    t = np.ascontiguousarray(np.asarray(t, dtype=np.float64))
    coef = np.zeros(3, np.float64)
    _check(lib().moe_fit_op_times(n.size, ctypes.c_void_p(n.ctypes.data), ctypes.c_void_p(U.ctypes.data),
                                  ctypes.c_void_p(t.ctypes.data), int(m), float(b), 0 if form == "slot" else 1,
                                  ctypes.c_void_p(coef.ctypes.data)), "moe_fit_op_times")
    return tuple(float(c) for c in coef)


# ---------------------------------------------------------------- FP8 (e4m3) experts
def quantize_rows_e4m3(src: torch.Tensor):
    """Row-wise e4m3 codes (uint8, same shape) and fp32 row scales of a 2-D or 3-D fp32/bf16
    CUDA tensor (rows = all leading dimensions)."""
    if (index := src.get_device()) >= 0 and index != _current_device():
        return _there(src, quantize_rows_e4m3, src)
    if src.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("quantize_rows_e4m3 takes fp32 or bf16")
    cols = src.shape[-1]
    rows = src.numel() // cols
    q = torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    scale = torch.empty(src.shape[:-1], dtype=torch.float32, device=src.device)
    _check(lib().moe_quantize_rows_e4m3(_dev(src, "src"), MOE_F32 if src.dtype == torch.float32 else MOE_BF16,
                                        rows, cols, ctypes.c_void_p(q.data_ptr()),
                                        ctypes.c_void_p(scale.data_ptr()), _stream(src.device)),
           "moe_quantize_rows_e4m3")
    return q, scale


def quantize_experts(weights):
    """(w_gate, w_up, w_down) bf16/fp32 -> (codes, row scales) for an e4m3 layer."""
    qs = [quantize_rows_e4m3(w) for w in weights]
    return tuple(q for q, _ in qs), tuple(s for _, s in qs)


def _scales(layer: Layer, scales) -> WeightScales:
    sg, su, sd = scales
    return WeightScales(_dev(sg, "s_gate", torch.float32, (layer.N, layer.f)),
                        _dev(su, "s_up", torch.float32, (layer.N, layer.f)),
                        _dev(sd, "s_down", torch.float32, (layer.N, layer.d)))


def expert_op_perslot_fp8(layer: Layer, weights, scales, xq: torch.Tensor, x_scale: torch.Tensor, ids: torch.Tensor,
                          gates: torch.Tensor, y=None, accumulate: bool = False, ws=None):
    """moe_expert_op_perslot_fp8: the per-slot form on e4m3 experts with row scales (the quantized experts of [Lan] App. E Table 6)."""
    if (index := xq.get_device()) >= 0 and index != _current_device():
        return _there(xq, expert_op_perslot_fp8, layer, weights, scales, xq, x_scale, ids, gates, y, accumulate, ws)
    n = xq.shape[0]
    ws = ws if ws is not None else workspace(layer, n, xq.device)
    y, yp = _y(layer, xq, y)
    sc = _scales(layer, scales)
    _check(lib().moe_expert_op_perslot_fp8(ctypes.byref(layer), *_weights(layer, weights), ctypes.byref(sc),
                                           _dev(xq, "x", torch.uint8, (n, layer.d)),
                                           _dev(x_scale, "x_scale", torch.float32, (n,)),
                                           _dev(ids, "ids", torch.int32, (n, layer.m)),
                                           _dev(gates, "gates", torch.float32, (n, layer.m)), n,
                                           int(bool(accumulate)), yp, ctypes.c_void_p(ws.data_ptr()),
                                           ws.numel(), _stream(xq.device)), "moe_expert_op_perslot_fp8")
    return y


def expert_op_dedup_ids_fp8(layer: Layer, weights, scales, xq: torch.Tensor, x_scale: torch.Tensor, ids: torch.Tensor,
                            gates: torch.Tensor, y=None, accumulate: bool = False, ws=None):
    """moe_expert_op_dedup_ids_fp8: the deduplicating form from ids on e4m3 experts, the grouping built in the kernel ([Lan] §1; App. E Table 6)."""
    if (index := xq.get_device()) >= 0 and index != _current_device():
        return _there(xq, expert_op_dedup_ids_fp8, layer, weights, scales, xq, x_scale, ids, gates, y, accumulate, ws)
    n = xq.shape[0]
    ws = ws if ws is not None else workspace(layer, n, xq.device)
    y, yp = _y(layer, xq, y)
    sc = _scales(layer, scales)
    _check(lib().moe_expert_op_dedup_ids_fp8(ctypes.byref(layer), *_weights(layer, weights), ctypes.byref(sc),
                                             _dev(xq, "x", torch.uint8, (n, layer.d)),
                                             _dev(x_scale, "x_scale", torch.float32, (n,)),
                                             _dev(ids, "ids", torch.int32, (n, layer.m)),
                                             _dev(gates, "gates", torch.float32, (n, layer.m)), n,
                                             int(bool(accumulate)), yp, ctypes.c_void_p(ws.data_ptr()),
                                             ws.numel(), _stream(xq.device)), "moe_expert_op_dedup_ids_fp8")
    return y


def expert_op_dedup_fp8(layer: Layer, weights, scales, xq: torch.Tensor, x_scale: torch.Tensor, gates: torch.Tensor,
                        grouping: Grouping, y=None, accumulate: bool = False, ws=None):
    """moe_expert_op_dedup_fp8: the deduplicating form on e4m3 experts and a precomputed grouping ([Lan] §1; App. E Table 6)."""
    if (index := xq.get_device()) >= 0 and index != _current_device():
        return _there(xq, expert_op_dedup_fp8, layer, weights, scales, xq, x_scale, gates, grouping, y, accumulate, ws)
    n = xq.shape[0]
    ws = ws if ws is not None else workspace(layer, n, xq.device)
    y, yp = _y(layer, xq, y)
    sc = _scales(layer, scales)
    _check(lib().moe_expert_op_dedup_fp8(ctypes.byref(layer), *_weights(layer, weights), ctypes.byref(sc),
                                         _dev(xq, "x", torch.uint8, (n, layer.d)),
                                         _dev(x_scale, "x_scale", torch.float32, (n,)),
                                         _dev(gates, "gates", torch.float32, (n, layer.m)), n,
                                         _dev(grouping.num_distinct, "num_distinct"),
                                         _dev(grouping.expert_list, "expert_list"),
                                         _dev(grouping.offsets, "offsets"),
                                         _dev(grouping.slot_order, "slot_order"),
                                         int(bool(accumulate)), yp, ctypes.c_void_p(ws.data_ptr()),
                                         ws.numel(), _stream(xq.device)), "moe_expert_op_dedup_fp8")
    return y


# ---------------------------------------------------------------- verify-side neighbours
def spec_accept(draft, q, p, r, u, greedy: bool = False, n_accepted=None, token=None):
    """One round of speculative sampling for B sequences ("Lossless but Not Free", §3.1,
    Algorithm 1) on the device.  draft int32 [B, K], q fp32 [B, K, V], p fp32 [B, K+1, V],
    r fp32 [B, K], u fp32 [B] (q, r, u may be None when greedy).  Returns (n_accepted, token),
    int32 [B] each."""
    if (index := p.get_device()) >= 0 and index != _current_device():
        return _there(p, spec_accept, draft, q, p, r, u, greedy, n_accepted, token)
    B, K1, V = p.shape
    K = K1 - 1
    dev = p.device
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if token is None:
        token = torch.empty(B, dtype=torch.int32, device=dev)
    dptr = lambda t, name, dt: None if t is None else _dev(t, name, dt)
    _check(lib().moe_spec_accept(dptr(draft, "draft", torch.int32) if K else None, dptr(q, "q", torch.float32),
                                 _dev(p, "p", torch.float32), dptr(r, "r", torch.float32), dptr(u, "u", torch.float32),
                                 B, K, V, int(bool(greedy)), _dev(n_accepted, "n_accepted", torch.int32),
                                 _dev(token, "token", torch.int32), _stream(dev)), "moe_spec_accept")
    return n_accepted, token


def union_cost(bitmaps, subsets, pv, bcoef, beta: float, out=None, ws=None):
    """SpecFit §3.2 eqs (3)-(5) on the device: bitmaps uint64-as-int64 [nodes+1, L, W], subsets
    int32/uint32 bits [S], pv float64 [nodes], bcoef float64 [nodes+1].  Returns dict(F, size,
    R, T, best) of device tensors."""
    if (index := bitmaps.get_device()) >= 0 and index != _current_device():
        return _there(bitmaps, union_cost, bitmaps, subsets, pv, bcoef, beta, out, ws)
    nodes1, L, W = bitmaps.shape
    S = subsets.numel()
    dev = bitmaps.device
    if out is None:
        out = dict(F=torch.empty(S, dtype=torch.int32, device=dev), size=torch.empty(S, dtype=torch.int32, device=dev),
                   R=torch.empty(S, dtype=torch.float64, device=dev), T=torch.empty(S, dtype=torch.float64, device=dev),
                   best=torch.empty(1, dtype=torch.int32, device=dev))
    if ws is None:
        ws = torch.empty(int(lib().moe_union_cost_workspace_bytes(S)), dtype=torch.uint8, device=dev)
    _check(lib().moe_union_cost(_dev(bitmaps, "bitmaps", torch.int64), nodes1 - 1, L, W,
                                _dev(subsets, "subsets", torch.int32), S,
                                _dev(pv, "pv", torch.float64) if nodes1 > 1 else None,
                                _dev(bcoef, "bcoef", torch.float64), float(beta),
                                _dev(out["F"], "F", torch.int32), _dev(out["size"], "size", torch.int32),
                                _dev(out["R"], "R", torch.float64), _dev(out["T"], "T", torch.float64),
                                _dev(out["best"], "best", torch.int32), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                _stream(dev)), "moe_union_cost")
    return out


def read_probe(buf: torch.Tensor, ws: torch.Tensor) -> int:
    """Enqueue the read-only streaming probe over buf (a CUDA tensor); returns the bytes it reads."""
    nbytes = buf.numel() * buf.element_size()
    _call("moe_read_probe", buf.device, ctypes.c_void_p(buf.data_ptr()), nbytes, ctypes.c_void_p(ws.data_ptr()),
          _stream(buf.device))
    return nbytes // 32768 * 32768


# ---------------------------------------------------------------- attention side of the pass
ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}
MAX_TREE_TOKENS = 64
_HEAD_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_CACHE_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.uint8: MOE_E4M3}
# Descriptors of these calls, which run once per layer and pass, are packed as bytes and passed by
# address: a fraction of a ctypes structure's cost.
_pack_heads = struct.Struct("@Pqqii").pack      # moe_heads_t
_pack_rotary = struct.Struct("@PPiiii").pack    # moe_rotary_t
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _device_of(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _heads(t: torch.Tensor, name: str, tokens: int, heads: int, dim: int, device: int) -> bytes:
    """The descriptor of a [tokens, heads, dim] tensor on `device`: any token and head strides, dense channels."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError(f"{name} must be a CUDA tensor on device {device}")
    code = _HEAD_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} must have shape {(tokens, heads, dim)}, got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError(f"{name} must have contiguous channels")
    return _pack_heads(t.data_ptr(), st, sh, heads, code)


def _flat(t: torch.Tensor, name: str, dtype, shape, device: int) -> int:
    """The address of a contiguous tensor of this type and shape on `device`."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError(f"{name} must be a CUDA tensor on device {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new_heads(x: torch.Tensor, tokens: int, heads: int, dim: int):
    """A dense [tokens, heads, dim] tensor of x's type beside it, and its descriptor."""
    y = torch.empty((tokens, heads, dim), dtype=x.dtype, device=x.device)
    return y, _pack_heads(y.data_ptr(), heads * dim, dim, heads, _HEAD_TYPES[x.dtype])


def _ws_ptr(ws, device: int):
    if ws is None:
        return None
    if ws.get_device() != device:
        raise TypeError(f"ws must be a CUDA tensor on device {device}")
    return ws.data_ptr()


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """moe_rope_frequencies: (rot / 2 frequencies as float64, magnitude) of a rotary table; scaling
    "plain", "linear", "base" or "by_parts" (the last needs `original`, the trained context)."""
    w = np.zeros(max(rot // 2, 1), np.float64)
    mag = ctypes.c_double(0.0)
    _check(lib().moe_rope_frequencies(int(rot), float(base), ROPE_SCALING[scaling], float(factor), int(original),
                                      float(beta_fast), float(beta_slow), ctypes.c_void_p(w.ctypes.data),
                                      ctypes.byref(mag)), "moe_rope_frequencies")
    return w, mag.value


def rope_table(positions: int, w, magnitude: float = 1.0, device=None) -> torch.Tensor:
    """moe_rope_table: fp32 [positions, rot / 2, 2] of m cos(p w_i), m sin(p w_i)."""
    w = np.ascontiguousarray(np.asarray(w, dtype=np.float64))
    table = torch.empty((positions, w.size, 2), dtype=torch.float32, device=device or "cuda")
    _call("moe_rope_table", table.device, ctypes.c_void_p(w.ctypes.data), w.size, float(magnitude), int(positions),
          ctypes.c_void_p(table.data_ptr()), _stream(table.device))
    return table


def _rotary(table: torch.Tensor, positions: torch.Tensor, tokens: int, interleaved: bool, inverse: bool, device: int) -> bytes:
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError(f"table must have shape (positions, rot / 2, 2), got {tuple(shape)}")
    return _pack_rotary(_flat(table, "table", torch.float32, shape, device),
                        _flat(positions, "positions", torch.int32, (tokens,), device),
                        shape[0], 2 * shape[1], 1 if interleaved else 0, 1 if inverse else 0)


def rope(q, k, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False, inverse: bool = False,
         q_out=None, k_out=None, ws=None):
    """moe_rope: rotates the rows of q [tokens, q heads, dim] and k [tokens, k heads, dim] (either may be
    None) by their positions; inverse gives the gradient's direction.  Returns (q_out, k_out); an output
    may be its input.  ws (any workspace) records positions beyond the table."""
    ref = q if q is not None else k
    device = _device_of(ref, "q" if q is not None else "k")
    if device != _current_device():
        return _there(ref, rope, q, k, positions, table, interleaved, inverse, q_out, k_out, ws)
    tokens, _, dim = ref.shape
    dq = dqo = dk = dko = None
    if q is not None:
        heads = q.shape[1]
        dq = _heads(q, "q", tokens, heads, dim, device)
        if q_out is None:
            q_out, dqo = _new_heads(q, tokens, heads, dim)
        else:
            dqo = _heads(q_out, "q_out", tokens, heads, dim, device)
    if k is not None:
        heads = k.shape[1]
        dk = _heads(k, "k", tokens, heads, dim, device)
        if k_out is None:
            k_out, dko = _new_heads(k, tokens, heads, dim)
        else:
            dko = _heads(k_out, "k_out", tokens, heads, dim, device)
    code = (_lib or lib()).moe_rope(dq, dqo, dk, dko, tokens, dim,
                                    _rotary(table, positions, tokens, interleaved, inverse, device),
                                    _ws_ptr(ws, device), _raw_stream(device))
    if code:
        raise MoeError(code, "moe_rope")
    return q_out, k_out


class KVCache:
    """A paged key/value cache (moe_kv_cache_t) over tensors the caller owns: k and v
    [pages, page, heads, dim] (fp32, bf16, or uint8 e4m3 codes; equal strides, dense channels), and
    for codes the scales fp32 [pages, heads, page]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale=None, v_scale=None):
        if not k.is_cuda or not v.is_cuda:
            raise TypeError("k and v must be CUDA tensors")
        code = _CACHE_TYPES.get(k.dtype)
        if code is None or v.dtype != k.dtype:
            raise TypeError(f"k and v must be float32, bfloat16 or uint8 alike, got {k.dtype} and {v.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or (k.stride(3) != 1 and k.shape[3] > 1):
            raise ValueError("k and v must have one shape (pages, page, heads, dim), equal strides and dense channels")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page, self.heads, self.dim = k.shape
        ks = vs = None
        if code == MOE_E4M3:
            shape = (self.pages, self.heads, self.page)
            ks = _dev(k_scale, "k_scale", torch.float32, shape)
            vs = _dev(v_scale, "v_scale", torch.float32, shape)
        elif k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to a cache of e4m3 codes")
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} must be on {k.device}, got {t.device}")
        self.desc = CacheDesc(k.data_ptr(), v.data_ptr(), ks, vs, *k.stride()[:3], code, self.heads, self.dim,
                              self.page, self.pages, 0)
        self.device, self.index = k.device, k.get_device()
        self.address = ctypes.addressof(self.desc)


def kv_cache(pages: int, page: int, heads: int, dim: int, dtype: str = "bf16", device=None) -> KVCache:
    """A zeroed cache of `pages` pages of `page` tokens: dtype "bf16", "f32" or "e4m3" (codes and scales)."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.uint8}[dtype]
    k, v = (torch.zeros((pages, page, heads, dim), dtype=t, device=device or "cuda") for _ in range(2))
    if dtype != "e4m3":
        return KVCache(k, v)
    return KVCache(k, v, *(torch.ones((pages, heads, page), dtype=torch.float32, device=k.device) for _ in range(2)))


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, q=None, positions=None, table=None,
             interleaved: bool = False, q_out=None, ws=None):
    """moe_kv_write: the rows k, v [tokens, heads, dim] into the cache's slots int32 [tokens] (a negative
    slot takes nothing), quantised for an e4m3 cache.  With positions and table the keys are rotated
    before, and q [tokens, q heads, dim], when given, is rotated into q_out, which is returned (None
    without q).  ws (any workspace) records slots and positions out of range."""
    device, dim = cache.index, cache.dim
    if device != _current_device():
        return _there(cache.k, kv_write, cache, k, v, slots, q, positions, table, interleaved, q_out, ws)
    tokens = k.shape[0]
    dk = _heads(k, "k", tokens, cache.heads, dim, device)
    dv = _heads(v, "v", tokens, cache.heads, dim, device)
    rot = dq = dqo = None
    if (table is None) != (positions is None):
        raise ValueError("rotation takes both positions and table")
    if table is not None:
        rot = _rotary(table, positions, tokens, interleaved, False, device)
    if q is not None:
        if table is None:
            raise ValueError("q is only rotated: it takes positions and table")
        heads = q.shape[1]
        dq = _heads(q, "q", tokens, heads, dim, device)
        if q_out is None:
            q_out, dqo = _new_heads(q, tokens, heads, dim)
        else:
            dqo = _heads(q_out, "q_out", tokens, heads, dim, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    code = (_lib or lib()).moe_kv_write(cache.address, dk, dv, _flat(slots, "slots", torch.int32, (tokens,), device), tokens,
                                        rot, dq, dqo, _ws_ptr(ws, device), _raw_stream(device))
    if code:
        raise MoeError(code, "moe_kv_write")
    return q_out


def kv_read(cache: KVCache, slots: torch.Tensor, dtype=torch.bfloat16, k_out=None, v_out=None, ws=None):
    """moe_kv_read: the cache's rows of slots int32 [tokens] as (k, v) [tokens, heads, dim], fp32 or bf16;
    zeros for a negative slot."""
    device = cache.index
    if device != _current_device():
        return _there(cache.k, kv_read, cache, slots, dtype, k_out, v_out, ws)
    tokens = slots.shape[0]
    shape = (tokens, cache.heads, cache.dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=cache.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=cache.device)
    code = (_lib or lib()).moe_kv_read(cache.address, _flat(slots, "slots", torch.int32, (tokens,), device), tokens,
                                       _heads(k_out, "k_out", *shape, device), _heads(v_out, "v_out", *shape, device),
                                       _ws_ptr(ws, device), _raw_stream(device))
    if code:
        raise MoeError(code, "moe_kv_read")
    return k_out, v_out


def tree_attention_workspace(cache: KVCache, tokens: int, seqs: int, q_heads: int) -> torch.Tensor:
    """A zeroed workspace for tree_attention calls of up to this many tokens and sequences."""
    with torch.cuda.device(cache.index):   # the size goes by its number of SMs
        nbytes = int(lib().moe_tree_attention_workspace_bytes(cache.address, tokens, seqs, q_heads))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    _call("moe_workspace_init", cache.device, ws.data_ptr(), nbytes, _stream(cache.device))
    return ws


def tree_attention(cache: KVCache, q: torch.Tensor, q_start: torch.Tensor, ctx: torch.Tensor, page_table: torch.Tensor,
                   mask=None, scale=None, max_tokens: int = MAX_TREE_TOKENS, out=None, lse=None,
                   return_lse: bool = False, ws=None):
    """moe_tree_attention: attention of drafted tokens over the cache.  q [tokens, q heads, dim] holds the
    tokens of all sequences, q_start int32 [seqs + 1] their bounds, ctx int32 [seqs] the cached positions
    before them, page_table int32 [seqs, max pages]; mask int64 [tokens], bit j of a token's word set
    where it sees drafted token j of its sequence (None: a chain); scale defaults to dim^-0.5.  Returns
    out, or (out, lse) with return_lse.

    max_tokens bounds a sequence's tokens and chooses the kernel: with max_tokens times the query heads of
    a key head at most 64, that for few rows, which is faster for them.  Without ws (tree_attention_workspace)
    each call allocates and clears one of tens of megabytes."""
    device, dim = cache.index, cache.dim
    if device != _current_device():
        return _there(cache.k, tree_attention, cache, q, q_start, ctx, page_table, mask, scale, max_tokens, out, lse, return_lse, ws)
    tokens, heads = q.shape[0], q.shape[1]
    seqs, max_pages = page_table.shape
    dq = _heads(q, "q", tokens, heads, dim, device)
    if out is None:
        out, do = _new_heads(q, tokens, heads, dim)
    else:
        do = _heads(out, "out", tokens, heads, dim, device)
    if return_lse and lse is None:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=cache.device)
    if ws is None:
        ws = tree_attention_workspace(cache, tokens, seqs, heads)
    code = (_lib or lib()).moe_tree_attention(
        cache.address, dq, do,
        None if lse is None else _flat(lse, "lse", torch.float32, (tokens, heads), device),
        _flat(q_start, "q_start", torch.int32, (seqs + 1,), device), _flat(ctx, "ctx", torch.int32, (seqs,), device),
        _flat(page_table, "page_table", torch.int32, (seqs, max_pages), device),
        None if mask is None else _flat(mask, "mask", torch.int64, (tokens,), device),
        seqs, tokens, max_tokens, max_pages, dim ** -0.5 if scale is None else scale,
        _ws_ptr(ws, device), ws.numel(), _raw_stream(device))
    if code:
        raise MoeError(code, "moe_tree_attention")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------- latent attention
class LatentCache:
    """A paged cache of latent rows (moe_latent_cache_t) over a tensor the caller owns: rows [pages, page,
    rank + rope] (fp32 or bf16, dense channels), the latent of a token in its first rank channels and its
    rotary key in the others."""

    def __init__(self, rows: torch.Tensor, rank: int):
        if not rows.is_cuda:
            raise TypeError("rows must be a CUDA tensor")
        code = _HEAD_TYPES.get(rows.dtype)
        if code is None:
            raise TypeError(f"rows must be float32 or bfloat16, got {rows.dtype}")
        if rows.dim() != 3 or rows.stride(2) != 1:
            raise ValueError("rows must have shape (pages, page, rank + rope) and dense channels")
        if not 0 < rank < rows.shape[2]:
            raise ValueError(f"rank must leave rotary channels of {rows.shape[2]}, got {rank}")
        self.rows, self.rank, self.rope = rows, rank, rows.shape[2] - rank
        self.pages, self.page = rows.shape[:2]
        self.desc = LatentDesc(rows.data_ptr(), *rows.stride()[:2], code, rank, self.rope, self.page, self.pages, 0)
        self.device, self.index = rows.device, rows.get_device()
        self.address = ctypes.addressof(self.desc)


def latent_cache(pages: int, page: int, rank: int, rope: int, dtype: str = "bf16", device=None) -> LatentCache:
    """A zeroed latent cache of `pages` pages of `page` tokens: dtype "bf16" or "f32"."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    return LatentCache(torch.zeros((pages, page, rank + rope), dtype=t, device=device or "cuda"), rank)


def _rows(t: torch.Tensor, name: str, tokens: int, dim: int, device: int) -> bytes:
    """The descriptor of a [tokens, dim] tensor on `device`: any token stride, dense channels."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError(f"{name} must be a CUDA tensor on device {device}")
    code = _HEAD_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.shape != (tokens, dim):
        raise ValueError(f"{name} must have shape {(tokens, dim)}, got {tuple(t.shape)}")
    st, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError(f"{name} must have contiguous channels")
    return _pack_heads(t.data_ptr(), st, 0, 1, code)


def latent_write(cache: LatentCache, latent: torch.Tensor, k_rope: torch.Tensor, slots: torch.Tensor, norm=None,
                 eps: float = 1e-6, q=None, positions=None, table=None, interleaved: bool = False, q_out=None, ws=None):
    """moe_latent_write: latents [tokens, rank] and rotary keys [tokens, rope] into the cache's slots int32
    [tokens] (a negative slot takes nothing).  With norm (fp32 [rank]) the latents are RMS-normalised and
    multiplied by it; with positions and table the rotary keys are rotated, and q [tokens, heads, rope], the
    queries' rotary channels, when given, into q_out, which is returned (None without q).  ws (any
    workspace) records slots and positions out of range."""
    device = cache.index
    if device != _current_device():
        return _there(cache.rows, latent_write, cache, latent, k_rope, slots, norm, eps, q, positions, table, interleaved, q_out, ws)
    tokens, rope = latent.shape[0], cache.rope
    dl = _rows(latent, "latent", tokens, cache.rank, device)
    dk = _rows(k_rope, "k_rope", tokens, rope, device)
    rot = dq = dqo = None
    if (table is None) != (positions is None):
        raise ValueError("rotation takes both positions and table")
    if table is not None:
        rot = _rotary(table, positions, tokens, interleaved, False, device)
    if q is not None:
        if table is None:
            raise ValueError("q is only rotated: it takes positions and table")
        heads = q.shape[1]
        dq = _heads(q, "q", tokens, heads, rope, device)
        if q_out is None:
            q_out, dqo = _new_heads(q, tokens, heads, rope)
        else:
            dqo = _heads(q_out, "q_out", tokens, heads, rope, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    code = (_lib or lib()).moe_latent_write(cache.address, dl, dk, _flat(slots, "slots", torch.int32, (tokens,), device), tokens,
                                            None if norm is None else _flat(norm, "norm", torch.float32, (cache.rank,), device),
                                            eps, rot, dq, dqo, _ws_ptr(ws, device), _raw_stream(device))
    if code:
        raise MoeError(code, "moe_latent_write")
    return q_out


def latent_attention_workspace(cache: LatentCache, tokens: int, seqs: int, heads: int) -> torch.Tensor:
    """A zeroed workspace for latent_attention calls of up to this many tokens and sequences."""
    with torch.cuda.device(cache.index):   # the size goes by its number of SMs
        nbytes = int(lib().moe_latent_attention_workspace_bytes(cache.address, tokens, seqs, heads))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    _call("moe_workspace_init", cache.device, ws.data_ptr(), nbytes, _stream(cache.device))
    return ws


def latent_attention(cache: LatentCache, q: torch.Tensor, q_start: torch.Tensor, ctx: torch.Tensor, page_table: torch.Tensor,
                     scale: float, mask=None, max_tokens: int = MAX_TREE_TOKENS, out=None, lse=None,
                     return_lse: bool = False, ws=None):
    """moe_latent_attention: attention of drafted tokens over a latent cache in the absorbed form.  q [tokens,
    heads, rank + rope] holds each head's query multiplied by its key matrix, and its rotary channels;
    q_start, ctx, page_table and mask are tree_attention's.  scale has no default: it goes by the width
    of the queries before they were multiplied.  Returns out [tokens, heads, rank], to be multiplied
    by each head's value matrix, or (out, lse) with return_lse.

    max_tokens bounds a sequence's tokens and chooses, with heads, how many rows a tile of the cache serves.
    Without ws (latent_attention_workspace) each call allocates and clears one of tens of megabytes."""
    device = cache.index
    if device != _current_device():
        return _there(cache.rows, latent_attention, cache, q, q_start, ctx, page_table, scale, mask, max_tokens, out, lse,
                      return_lse, ws)
    tokens, heads = q.shape[0], q.shape[1]
    seqs, max_pages = page_table.shape
    dq = _heads(q, "q", tokens, heads, cache.rank + cache.rope, device)
    if out is None:
        out, do = _new_heads(q, tokens, heads, cache.rank)
    else:
        do = _heads(out, "out", tokens, heads, cache.rank, device)
    if return_lse and lse is None:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=cache.device)
    if ws is None:
        ws = latent_attention_workspace(cache, tokens, seqs, heads)
    code = (_lib or lib()).moe_latent_attention(
        cache.address, dq, do,
        None if lse is None else _flat(lse, "lse", torch.float32, (tokens, heads), device),
        _flat(q_start, "q_start", torch.int32, (seqs + 1,), device), _flat(ctx, "ctx", torch.int32, (seqs,), device),
        _flat(page_table, "page_table", torch.int32, (seqs, max_pages), device),
        None if mask is None else _flat(mask, "mask", torch.int64, (tokens,), device),
        seqs, tokens, max_tokens, max_pages, scale, _ws_ptr(ws, device), ws.numel(), _raw_stream(device))
    if code:
        raise MoeError(code, "moe_latent_attention")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------- pages of a cache
class PagePool:
    """The pages of some layers' caches (KVCache or LatentCache, equal numbers of pages and tokens a page, none
    twice) and who holds them (moe_page_pool_t), over tensors the caller owns: refs int32 [pages] (holders of a page),
    table int32 [seqs, max pages] (the page_table of the attention calls), held int32 [seqs] (pages a
    sequence holds).  All zero: every page is free.  ws is the calls' workspace; its error word records
    ids, lengths and paths out of range."""

    def __init__(self, caches, refs: torch.Tensor, table: torch.Tensor, held: torch.Tensor):
        self.caches, self.refs, self.table, self.held = list(caches), refs, table, held
        if not self.caches:
            raise ValueError("a pool needs a cache")
        for c in self.caches:
            if not isinstance(c, (KVCache, LatentCache)):
                raise TypeError("caches must be KVCache or LatentCache")
        first = self.caches[0]
        self.pages, self.page, self.device, self.index = first.pages, first.page, first.device, first.index
        for c in self.caches:
            if (c.pages, c.page, c.index) != (self.pages, self.page, self.index):
                raise ValueError("caches must have equal pages and lie on one device")
        parts = [t.data_ptr() for c in self.caches for t in ((c.k, c.v) if isinstance(c, KVCache) else (c.rows,))]
        if len(set(parts)) < len(parts):
            raise ValueError("caches must not share memory: rows would move twice")
        index = self.index
        _flat(refs, "refs", torch.int32, (self.pages,), index)
        if table.dim() != 2:
            raise ValueError("table must have shape (seqs, max pages)")
        self.seqs, self.max_pages = table.shape
        self.desc = PoolDesc(refs.data_ptr(), _flat(table, "table", torch.int32, table.shape, index),
                             _flat(held, "held", torch.int32, (self.seqs,), index), self.pages, self.page, self.seqs, self.max_pages)
        kv = [c.desc for c in self.caches if isinstance(c, KVCache)]
        latent = [c.desc for c in self.caches if isinstance(c, LatentCache)]
        self._kv, self._latent = (CacheDesc * max(len(kv), 1))(*kv), (LatentDesc * max(len(latent), 1))(*latent)
        self._caches = CachesDesc(ctypes.addressof(self._kv), ctypes.addressof(self._latent), len(kv), len(latent))
        self.address, self.caches_address = ctypes.addressof(self.desc), ctypes.addressof(self._caches)
        self.ws_bytes = int(lib().moe_pages_workspace_bytes(self.address))
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        _call("moe_workspace_init", self.device, self.ws.data_ptr(), self.ws_bytes, _stream(self.device))


def page_pool(caches, seqs: int, max_pages: int) -> PagePool:
    """A pool over these caches with every page free."""
    caches = list(caches)
    z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=caches[0].device)
    return PagePool(caches, z(caches[0].pages), z(seqs, max_pages), z(seqs))


def pages_reserve(pool: PagePool, length: torch.Tensor, need: torch.Tensor, got=None) -> torch.Tensor:
    """moe_pages_reserve: pages for need int32 [seqs] more tokens of every sequence after its length int32 [seqs],
    the lowest free ones, sequences in order; a shared page that would be written is copied in every
    cache, or replaced where it lies behind the length.  Returns got int32 [seqs]: 1 where the sequence has its pages, 0 where they ran out."""
    device = pool.index
    if device != _current_device():
        return _there(pool.refs, pages_reserve, pool, length, need, got)
    shape = (pool.seqs,)
    if got is None:
        got = torch.empty(shape, dtype=torch.int32, device=pool.device)
    code = (_lib or lib()).moe_pages_reserve(pool.address, _flat(length, "length", torch.int32, shape, device),
                                             _flat(need, "need", torch.int32, shape, device),
                                             _flat(got, "got", torch.int32, shape, device), pool.caches_address,
                                             pool.ws.data_ptr(), pool.ws_bytes, _raw_stream(device))
    if code:
        raise MoeError(code, "moe_pages_reserve")
    return got


def pages_fork(pool: PagePool, src: torch.Tensor, dst: torch.Tensor, length: torch.Tensor) -> None:
    """moe_pages_fork: sequences dst int32 [n], which hold nothing, share the pages of sequences src int32 [n] and
    take their length (length int32 [seqs] is read and written)."""
    device = pool.index
    if device != _current_device():
        return _there(pool.refs, pages_fork, pool, src, dst, length)
    n = src.shape[0]
    code = (_lib or lib()).moe_pages_fork(pool.address, _flat(src, "src", torch.int32, (n,), device),
                                          _flat(dst, "dst", torch.int32, (n,), device), n,
                                          _flat(length, "length", torch.int32, (pool.seqs,), device),
                                          pool.ws.data_ptr(), pool.ws_bytes, _raw_stream(device))
    if code:
        raise MoeError(code, "moe_pages_fork")


def pages_accept(pool: PagePool, ctx: torch.Tensor, path, count: torch.Tensor, after=None) -> torch.Tensor:
    """moe_pages_accept: of the tokens drafted behind ctx int32 [seqs] those path int32 [seqs, max path] names (ascending,
    the first count int32 [seqs] of a row; None: the first ones) are kept: their rows become consecutive
    in every cache, pages behind them are given up.  A negative count leaves a sequence alone.  Returns
    after int32 [seqs], the new lengths (may be ctx itself)."""
    device = pool.index
    if device != _current_device():
        return _there(pool.refs, pages_accept, pool, ctx, path, count, after)
    shape = (pool.seqs,)
    if after is None:
        after = torch.empty(shape, dtype=torch.int32, device=pool.device)
    if path is not None and path.dim() != 2:
        raise ValueError("path must have shape (seqs, max path)")
    most = MAX_TREE_TOKENS if path is None else path.shape[1]
    code = (_lib or lib()).moe_pages_accept(pool.address, _flat(ctx, "ctx", torch.int32, shape, device),
                                            None if path is None else _flat(path, "path", torch.int32, (pool.seqs, most), device),
                                            _flat(count, "count", torch.int32, shape, device), most,
                                            _flat(after, "after", torch.int32, shape, device), pool.caches_address,
                                            pool.ws.data_ptr(), pool.ws_bytes, _raw_stream(device))
    if code:
        raise MoeError(code, "moe_pages_accept")
    return after


def pages_free(pool: PagePool, ids: torch.Tensor, length=None) -> None:
    """moe_pages_free: sequences ids int32 [n] (negative: none) give up their pages; length int32 [seqs], when given,
    becomes 0 for them."""
    device = pool.index
    if device != _current_device():
        return _there(pool.refs, pages_free, pool, ids, length)
    n = ids.shape[0]
    code = (_lib or lib()).moe_pages_free(pool.address, _flat(ids, "ids", torch.int32, (n,), device), n,
                                          None if length is None else _flat(length, "length", torch.int32, (pool.seqs,), device),
                                          pool.ws.data_ptr(), pool.ws_bytes, _raw_stream(device))
    if code:
        raise MoeError(code, "moe_pages_free")

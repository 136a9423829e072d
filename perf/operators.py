"""The attention side of a verification pass, as it is measured: rotary positions, the write of
the pass's keys and values into a paged cache (quantised or not), the read back, and attention of
a tree of drafted tokens over the cache.

``run`` computes each operator in its plain form (32-bit torch arithmetic, rounded once at the
end), or, where ``own`` is true, calls the library.

Definitions, for token t, head h and channel c:

* rotary: a table [positions][rot / 2][2] holds m cos(p w_i) and m sin(p w_i); the pair (a, b) of
  channels (i, i + rot / 2), or (2 i, 2 i + 1) in the interleaved layout, becomes
  (a cos - b sin, b cos + a sin), and under ``inverse``, the gradient's direction,
  (a cos + b sin, b cos - a sin).  Channels from rot on stay as they are.
* write: slot s of the cache is row s % page of page s / page; a negative slot takes nothing.  An
  e4m3 row of one head holds codes of x / scale, scale = max|x| / 448 (1 for a zero row).
* read: the rows of given slots, multiplied by their scales; zeros for a negative slot.
* attention: drafted token i of a sequence with ctx cached tokens sees cache positions [0, ctx),
  and position ctx + j where bit j of its mask is set; softmax over what it sees, 0 and a
  log-sum-exp of -inf where it sees nothing.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one pass of a 15-token draft and its root in a decoder layer: 32 query and 4 key heads
        {"name": "rope-verify-pass", "op": "rope", "tokens": 16, "q_heads": 32, "kv_heads": 4, "dim": 128, "rot": 128,
         "interleaved": False, "inverse": False, "type": "bf16", "positions": 40960},
        # the gradient's direction over a training batch, half of each head rotated, adjacent pairs
        {"name": "rope-grad-16381", "op": "rope", "tokens": 16381, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 64,
         "interleaved": True, "inverse": True, "type": "bf16", "positions": 131072},
        # a verification pass of one sequence: queries and keys rotated, keys and values quantised
        {"name": "write-verify-e4m3", "op": "write", "tokens": 16, "q_heads": 32, "kv_heads": 4, "dim": 128,
         "rot": 128, "interleaved": False, "type": "bf16", "cache": "e4m3", "page": 16, "positions": 40960},
        # a prompt written to the quantised cache, its keys rotated before
        {"name": "write-prompt-e4m3", "op": "write", "tokens": 16300, "q_heads": 0, "kv_heads": 8, "dim": 128,
         "rot": 0, "interleaved": False, "type": "bf16", "cache": "e4m3", "page": 64, "positions": 0},
        # a prompt chunk with everything in one call: rotation of all heads, a bf16 cache
        {"name": "write-rotary-bf16", "op": "write", "tokens": 8190, "q_heads": 32, "kv_heads": 4, "dim": 128,
         "rot": 128, "interleaved": False, "type": "bf16", "cache": "bf16", "page": 32, "positions": 40960},
        # a short prefix read back
        {"name": "read-prefix-e4m3", "op": "read", "tokens": 700, "kv_heads": 4, "dim": 128, "type": "bf16",
         "cache": "e4m3", "page": 16},
        # a long context read back whole
        {"name": "read-context-e4m3", "op": "read", "tokens": 131000, "kv_heads": 8, "dim": 128, "type": "bf16",
         "cache": "e4m3", "page": 64},
        # the smallest call: one sequence, one token, a short context; latency counts
        {"name": "attention-single-token", "op": "attention", "seqs": 1, "tokens": 1, "tree": False, "ctx_min": 300,
         "ctx_max": 300, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 16, "cache": "bf16"},
        # a serving batch with short chains of drafts and ragged contexts, quantised cache
        {"name": "attention-chains-e4m3", "op": "attention", "seqs": 16, "tokens": 5, "tree": False, "ctx_min": 801,
         "ctx_max": 4099, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cache": "e4m3"},
        # draft trees of the largest pass, 64 nodes, 8 query heads to a key head
        {"name": "attention-trees-64", "op": "attention", "seqs": 8, "tokens": 64, "tree": True, "ctx_min": 4001,
         "ctx_max": 8201, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 32, "cache": "bf16"},
        # two long contexts, one 16-token tree each
        {"name": "attention-long-bf16", "op": "attention", "seqs": 2, "tokens": 16, "tree": True, "ctx_min": 100003,
         "ctx_max": 131071, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 256, "cache": "bf16"},
        # long contexts in the quantised cache
        {"name": "attention-long-e4m3", "op": "attention", "seqs": 4, "tokens": 8, "tree": True, "ctx_min": 60001,
         "ctx_max": 65537, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cache": "e4m3"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "write", "read", "attention", "attention", "attention"))
    kv = rng.choice((1, 2, 4, 8))
    q = kv * rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128))
    if op == "rope":
        rot = rng.choice((dim, dim // 2, dim - 16))
        kind = rng.choice(("bf16", "bf16", "f32"))
        tokens = _log(rng, 1, min(16381, 16381 * 40 * 128 * 2 // ((q + kv) * dim * _BYTES[kind])))
        return {"op": op, "tokens": tokens, "q_heads": q, "kv_heads": kv, "dim": dim, "rot": rot,
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5, "type": kind, "positions": 40960}
    if op == "write":
        rotary = rng.random() < 0.6
        return {"op": op, "tokens": _log(rng, 1, 16300 if q <= 32 else 8190), "q_heads": q if rotary else 0, "kv_heads": kv,
                "dim": dim, "rot": rng.choice((dim, dim // 2)) if rotary else 0, "interleaved": rng.random() < 0.3,
                "type": rng.choice(("bf16", "f32")) if q <= 16 else "bf16", "cache": rng.choice(("bf16", "e4m3", "e4m3")),
                "page": rng.choice((16, 32, 64, 128)), "positions": 40960 if rotary else 0}
    if op == "read":
        return {"op": op, "tokens": _log(rng, 1, 131000), "kv_heads": kv, "dim": dim, "type": rng.choice(("bf16", "bf16", "f32")) if kv <= 4 else "bf16",
                "cache": rng.choice(("bf16", "e4m3", "e4m3")), "page": rng.choice((16, 32, 64, 128))}
    seqs, tokens = _log(rng, 1, 32), _log(rng, 1, 64)
    most = min(131071, 262144 * 4 // (seqs * kv), 9 * 10 ** 9 // (seqs * tokens * q * dim))
    ctx = _log(rng, 1, max(1, most))
    return {"op": op, "seqs": seqs, "tokens": tokens, "tree": rng.random() < 0.6, "ctx_min": rng.randint(0, ctx), "ctx_max": ctx,
            "q_heads": q, "kv_heads": kv, "dim": dim, "page": rng.choice((16, 32, 64, 128)), "cache": rng.choice(("bf16", "e4m3"))}


def _lens(c):
    """Cached and drafted tokens of each sequence: set by the case, not by the seed."""
    r = random.Random(c["seqs"] * 7919 + c["ctx_max"])
    ctx = [r.randint(c["ctx_min"], c["ctx_max"]) for _ in range(c["seqs"])]
    ctx[-1] = c["ctx_max"]
    n = [c["tokens"] if r.random() < 0.75 else r.randint(1, c["tokens"]) for _ in range(c["seqs"])]
    n[-1] = c["tokens"]
    return ctx, n


def work(c):
    if c["op"] == "rope":
        rows = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return {"bytes": 2 * rows * c["dim"] * _BYTES[c["type"]] + c["tokens"] * (4 + 4 * c["rot"]), "flops": 3 * rows * c["rot"]}
    if c["op"] == "write":
        rows, qrows = 2 * c["tokens"] * c["kv_heads"], c["tokens"] * c["q_heads"]
        b = rows * c["dim"] * (_BYTES[c["type"]] + _BYTES[c["cache"]]) + 2 * qrows * c["dim"] * _BYTES[c["type"]] + 4 * c["tokens"]
        if c["cache"] == "e4m3":
            b += 4 * rows
        if c["rot"]:
            b += c["tokens"] * (4 + 4 * c["rot"])
        return {"bytes": b, "flops": 3 * (qrows + rows // 2) * c["rot"] + 3 * rows * c["dim"] * (c["cache"] == "e4m3")}
    if c["op"] == "read":
        rows = 2 * c["tokens"] * c["kv_heads"]
        return {"bytes": rows * (c["dim"] * (_BYTES[c["type"]] + _BYTES[c["cache"]]) + 4 * (c["cache"] == "e4m3")) + 4 * c["tokens"],
                "flops": rows * c["dim"]}
    ctx, n = _lens(c)
    per = 2 * c["kv_heads"] * (c["dim"] * _BYTES[c["cache"]] + 4 * (c["cache"] == "e4m3"))
    kv = sum(a + b for a, b in zip(ctx, n))
    return {"bytes": per * kv + sum(n) * c["q_heads"] * (4 * c["dim"] + 4),
            "flops": sum(4 * b * c["q_heads"] * c["dim"] * (a + b) for a, b in zip(ctx, n))}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(c):
    """m cos and m sin of every position and frequency, base 1,000,000, positions stretched 4-fold
    beyond a third of the frequencies as long contexts are."""
    half = c["rot"] // 2
    w = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    w = torch.where(torch.arange(half, device="cuda") >= 2 * half // 3, w / 4, w)
    a = torch.arange(c["positions"], dtype=torch.float64, device="cuda")[:, None] * w
    return torch.stack((a.cos(), a.sin()), -1).mul_(0.1 * math.log(4.0) + 1).float()


def _cache(c, pages, g):
    """Pages full of what earlier tokens left, one page beyond the cache's own, and scales."""
    shape = (pages + 1, c["page"], c["kv_heads"], c["dim"])
    if c["cache"] != "e4m3":
        return [torch.randn(shape, generator=g, device="cuda", dtype=_TYPES[c["cache"]]) for _ in range(2)] + [None, None]
    # codes of N(0, 1) rows whose largest magnitudes lie near 448
    codes = [torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(130).clamp_(-448, 448)
             .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    scales = [torch.rand((pages + 1, c["kv_heads"], c["page"]), generator=g, device="cuda").mul_(0.004).add_(0.006) for _ in range(2)]
    return codes + scales


def _heads(c, heads, g):
    """[tokens, heads, dim] views of one projection's output, as a layer hands them on."""
    total = sum(heads)
    x = torch.randn((c["tokens"], total, c["dim"]), generator=g, device="cuda", dtype=_TYPES[c["type"]])
    return list(x.split(heads, 1))


def prepare(case, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    s = {"case": case, "op": case["op"]}
    c = case
    if c["op"] == "rope":
        s["q"], s["k"] = _heads(c, [c["q_heads"], c["kv_heads"]], g)
        start = int(rng.integers(0, c["positions"] - c["tokens"] + 1))
        s["positions"] = torch.arange(start, start + c["tokens"], dtype=torch.int32, device="cuda")
        s["table"] = _table(c)
        return s
    if c["op"] in ("write", "read"):
        pages = -(-c["tokens"] // c["page"]) + 3
        order = torch.from_numpy(rng.permutation(pages)).cuda()
        t = torch.arange(c["tokens"], device="cuda")
        slots = order[t // c["page"]] * c["page"] + t % c["page"]
        if c["tokens"] > 4:   # the padding of a batch's last rows
            slots[-2:] = -1
        s["slots"] = slots.int()
        s["k"], s["v"], s["k_scale"], s["v_scale"] = _cache(c, pages, g)
        if c["op"] == "write":
            heads = ([c["q_heads"]] if c["q_heads"] else []) + [c["kv_heads"]] * 2
            *q, s["new_k"], s["new_v"] = _heads(c, heads, g)
            s["q"] = q[0] if q else None
            if c["rot"]:
                start = int(rng.integers(0, c["positions"] - c["tokens"] + 1))
                s["positions"] = torch.arange(start, start + c["tokens"], dtype=torch.int32, device="cuda")
                s["table"] = _table(c)
        pages_own = pages
    else:
        ctx, n = _lens(c)
        need = [-(-(a + b) // c["page"]) for a, b in zip(ctx, n)]
        pages_own = sum(need) + 3
        order, at = rng.permutation(pages_own).astype(np.int32), 0
        table = np.zeros((len(ctx), max(need)), np.int32)
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        masks = []
        for k in n:
            seen = []
            for i in range(k):
                parent = i - 1 if not c["tree"] else int(rng.integers(max(0, i - 6), i)) if i else -1
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
            masks += seen
        s["mask"] = torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda() if c["tree"] else None
        s["page_table"] = torch.from_numpy(table).cuda()
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        s["k"], s["v"], s["k_scale"], s["v_scale"] = _cache(c, pages_own, g)
        # queries whose scores spread over several units, so that some keys stand out
        s["q"] = torch.randn((sum(n), c["q_heads"], c["dim"]), generator=g, device="cuda", dtype=torch.bfloat16).mul_(2)
    if own:
        from moe_speculative_decoding_gb300 import api
        cut = lambda x: None if x is None else x[:pages_own]
        s["cache"] = api.KVCache(cut(s["k"]), cut(s["v"]), cut(s["k_scale"]), cut(s["v_scale"]))
        if c["op"] == "attention":
            s["ws"] = api.tree_attention_workspace(s["cache"], s["q"].shape[0], c["seqs"], c["q_heads"])
    return s


# ---------------------------------------------------------------- the library's calls

def _call(s):
    from moe_speculative_decoding_gb300 import api
    c = s["case"]
    if s["op"] == "rope":
        return api.rope(s["q"], s["k"], s["positions"], s["table"], interleaved=c["interleaved"], inverse=c["inverse"])
    if s["op"] == "write":
        if c["rot"]:
            q = api.kv_write(s["cache"], s["new_k"], s["new_v"], s["slots"], q=s["q"], positions=s["positions"],
                             table=s["table"], interleaved=c["interleaved"])
        else:
            q = api.kv_write(s["cache"], s["new_k"], s["new_v"], s["slots"])
        return _written(s, q)
    if s["op"] == "read":
        return api.kv_read(s["cache"], s["slots"], dtype=_TYPES[c["type"]])
    return api.tree_attention(s["cache"], s["q"], s["starts"], s["ctx"], s["page_table"], mask=s["mask"],
                              max_tokens=c["tokens"], return_lse=True, ws=s["ws"])


def _written(s, q):
    """The cache after a write: codes as the 8-bit floats they are."""
    seen = [x[:-1].view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x[:-1] for x in (s["k"], s["v"])]
    seen += [s[x][:-1] for x in ("k_scale", "v_scale") if s[x] is not None]
    return seen + ([q] if q is not None else [])


# ---------------------------------------------------------------- plain forms

def _rotate(x, positions, table, c, inverse=False):
    x, rot = x.float(), c["rot"]
    t = table[positions.long()][:, None]
    cos, sin = t[..., 0], t[..., 1]
    if inverse:
        sin = -sin
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _store(s, name, x):
    c, buf = s["case"], s[name]
    slots = s["slots"].long()
    slots = torch.where(slots < 0, (buf.shape[0] - 1) * c["page"], slots)   # the page beyond the cache
    at, row = slots // c["page"], slots % c["page"]
    if c["cache"] != "e4m3":
        buf[at, row] = x.to(buf.dtype)
        return
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    buf.view(torch.float8_e4m3fn)[at, row] = (x / scale[..., None]).to(torch.float8_e4m3fn)
    s[name + "_scale"][at, :, row] = scale


def _values(s, name, pages):
    """The given pages' rows in 32 bits: [..., page, heads, dim]."""
    x = s[name][pages]
    if x.dtype != torch.uint8:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * s[name + "_scale"][pages].transpose(-1, -2)[..., None]


def _fetch(s, name):
    c, slots = s["case"], s["slots"].long()
    at, row = slots.clamp(min=0) // c["page"], slots.clamp(min=0) % c["page"]
    x = s[name][at, row]
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn).float() * s[name + "_scale"][at, :, row][..., None]
    return torch.where(slots[:, None, None] < 0, torch.zeros((), device=x.device), x.float()).to(_TYPES[c["type"]])


def _attend(s):
    c, q, starts, ctx = s["case"], s["q"], s["starts"].long(), s["ctx"].long()
    total, seqs, n, hk = q.shape[0], c["seqs"], c["tokens"], c["kv_heads"]
    token = torch.arange(total, device=q.device)
    b = torch.searchsorted(starts, token, right=True) - 1
    i = token - starts[b]
    rows = (starts[:-1, None] + torch.arange(n, device=q.device)).clamp(max=total - 1)
    x = q[rows].float().view(seqs, n, hk, -1, c["dim"]).transpose(1, 2).reshape(seqs, hk, -1, c["dim"])
    k = _values(s, "k", s["page_table"].long()).flatten(1, 2).transpose(1, 2)
    v = _values(s, "v", s["page_table"].long()).flatten(1, 2).transpose(1, 2)
    scores = x @ k.transpose(-1, -2) * c["dim"] ** -0.5
    drafted = torch.arange(k.shape[2], device=q.device) - ctx[:, None]
    if s["mask"] is None:
        seen = drafted[:, None] <= torch.arange(n, device=q.device)[:, None]
    else:
        seen = (s["mask"][rows][..., None] >> drafted.clamp(0, 63)[:, None] & 1 > 0) | (drafted[:, None] < 0)
    seen = seen & (drafted < (starts[1:] - starts[:-1])[:, None])[:, None]
    scores = scores.view(seqs, hk, n, -1, k.shape[2]).masked_fill(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (scores - top).exp()
    z = e.sum(-1, keepdim=True)
    out = (e.flatten(2, 3) @ v).view(*e.shape[:-1], c["dim"]) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (z.log() + top)[..., 0]
    return out.transpose(1, 2).flatten(2, 3)[b, i].to(q.dtype), lse.transpose(1, 2).flatten(2, 3)[b, i]


def run(s):
    if own:
        return _call(s)
    c = s["case"]
    if s["op"] == "rope":
        return tuple(_rotate(x, s["positions"], s["table"], c, c["inverse"]).to(x.dtype) for x in (s["q"], s["k"]))
    if s["op"] == "write":
        q, k = s["q"], s["new_k"].float()
        if c["rot"]:
            k = _rotate(k, s["positions"], s["table"], c)
            q = _rotate(q, s["positions"], s["table"], c).to(q.dtype)
        _store(s, "k", k)
        _store(s, "v", s["new_v"].float())
        return _written(s, q)
    if s["op"] == "read":
        return _fetch(s, "k"), _fetch(s, "v")
    return _attend(s)


# ---------------------------------------------------------------- in 64 bits

def _turned(x, s, c, sign):
    """Rotation as the product of each pair, taken as a complex number, with m e^(+-i angle)."""
    x = x.double()
    half = c["rot"] // 2
    t = s["table"].double()[s["positions"].long()]
    turn = torch.complex(t[..., 0], sign * t[..., 1])[:, None]
    y = x.clone()
    if c["interleaved"]:
        z = torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:2], half, 2).contiguous()) * turn
        y[..., :c["rot"]] = torch.view_as_real(z).reshape(*x.shape[:2], c["rot"])
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:c["rot"]].contiguous()) * turn
        y[..., :half], y[..., half:c["rot"]] = z.real, z.imag
    return y


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rope":
        return tuple(_turned(s[x], s, c, -1.0 if c["inverse"] else 1.0) for x in "qk")
    where = s["slots"].long() if c["op"] != "attention" else None
    if c["op"] == "write":
        keep = where >= 0
        at, row = where[keep] // c["page"], where[keep] % c["page"]
        rows = {"k": _turned(s["new_k"], s, c, 1.0) if c["rot"] else s["new_k"].double(), "v": s["new_v"].double()}
        caches, scales = [], []
        for name in "kv":
            x = rows[name][keep]
            if c["cache"] != "e4m3":
                old = s[name][:-1].double()
                old[at, row] = x
            else:
                old = s[name][:-1].view(torch.float8_e4m3fn).double()
                scale = x.abs().amax(-1) / 448
                scale[scale == 0] = 1
                old[at, row] = x / scale[..., None]
                kept = s[name + "_scale"][:-1].double()
                kept[at, :, row] = scale
                scales.append(kept)
            caches.append(old)
        return caches + scales + ([_turned(s["q"], s, c, 1.0)] if c["rot"] else [])
    if c["op"] == "read":
        found = []
        for name in "kv":
            x = torch.zeros((c["tokens"], c["kv_heads"], c["dim"]), dtype=torch.float64, device="cuda")
            keep = where >= 0
            at, row = where[keep] // c["page"], where[keep] % c["page"]
            y = s[name][at, row]
            if c["cache"] == "e4m3":
                y = y.view(torch.float8_e4m3fn).double() * s[name + "_scale"][at, :, row].double()[..., None]
            x[keep] = y.double()
            found.append(x)
        return tuple(found)
    if work(c)["flops"] > 2e11:
        return None
    group, outs, lses = c["q_heads"] // c["kv_heads"], [], []
    starts, ctx = s["starts"].tolist(), s["ctx"].tolist()
    masks = s["mask"].tolist() if s["mask"] is not None else None
    for b in range(c["seqs"]):
        n = starts[b + 1] - starts[b]
        pages = s["page_table"][b, :-(-(ctx[b] + n) // c["page"])].long()
        see = np.ones((n, ctx[b] + n), bool)
        for i in range(n):
            for j in range(n):
                see[i, ctx[b] + j] = j <= i if masks is None else (masks[starts[b] + i] >> j) & 1
        see = torch.from_numpy(see).cuda()
        out = torch.zeros((n, c["q_heads"], c["dim"]), dtype=torch.float64, device="cuda")
        lse = torch.zeros((n, c["q_heads"]), dtype=torch.float64, device="cuda")
        for h in range(c["kv_heads"]):
            kv = []
            for name in "kv":
                x = s[name][pages, :, h]
                if x.dtype == torch.uint8:
                    x = x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][pages, h].double()[..., None]
                kv.append(x.double().flatten(0, 1)[:ctx[b] + n])
            for j in range(group):
                a = s["q"][starts[b]:starts[b + 1], h * group + j].double() @ kv[0].T / math.sqrt(c["dim"])
                a = a.masked_fill(~see, -math.inf)
                lse[:, h * group + j] = torch.logsumexp(a, -1)
                out[:, h * group + j] = torch.softmax(a, -1) @ kv[1]
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)

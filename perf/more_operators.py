"""Latent attention and page management of a verification pass, as they are measured: the write of
compressed latents into a paged cache, attention of drafted tokens over it in the absorbed form, and
the steps that share, copy, compact and free the pages of every layer's cache.

``run`` computes each operator in its plain form (32-bit torch arithmetic, rounded once at the
end), or, where ``own`` is true, calls the library.

Definitions:

* latent write: a token's cache row is [y | r], y = c w / sqrt(mean(c^2) + eps) over its rank channels
  (c itself without w), r its rotary channels, each pair turned by the token's position; the rotary
  channels of its queries are turned likewise.  A negative slot takes nothing.
* latent attention: all heads read one row a position.  s = scale <q, row> over all channels,
  out = sum_p softmax(s)_p y_p over the rank channels; drafted token i of a sequence with ctx cached
  tokens sees [0, ctx), and ctx + j where bit j of its mask is set (without a mask, j <= i).
* pages: refs holds each page's holders (0: free), table a sequence's pages, held their number.
  free: a sequence gives its pages up.  fork: a sequence takes another's pages, each with one holder
  more.  reserve: sequences, in order, take the lowest free pages until they hold
  ceil((length + need) / page); a shared page with rows to keep that is about to be written is replaced
  by a copy, unless all its other holders have just done so; from the first sequence on whose
  pages are not there, none that needs some gets any (got = 0).  accept: row ctx + path[i] moves to ctx + i in every
  layer, the sequence then holds ceil((ctx + count) / page) pages and gives up the others.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
_EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one pass of a 15-token draft and its root in a layer with 16 heads
        {"name": "latent-write-pass", "op": "write", "tokens": 16, "heads": 16, "rank": 512, "rope": 64, "norm": True,
         "interleaved": True, "type": "bf16", "page": 64, "positions": 40960},
        # a batch of prompts written at once, many heads
        {"name": "latent-write-prompts", "op": "write", "tokens": 16301, "heads": 32, "rank": 512, "rope": 64, "norm": True,
         "interleaved": True, "type": "bf16", "page": 64, "positions": 131072},
        # the smallest call: one sequence, one token, a short context; latency counts
        {"name": "latent-single-token", "op": "attention", "seqs": 1, "tokens": 1, "tree": False, "ctx_min": 300,
         "ctx_max": 300, "heads": 16, "rank": 512, "rope": 64, "page": 64},
        # a serving batch, one token a sequence, ragged contexts
        {"name": "latent-decode-64", "op": "attention", "seqs": 64, "tokens": 1, "tree": False, "ctx_min": 801,
         "ctx_max": 8209, "heads": 16, "rank": 512, "rope": 64, "page": 64},
        # draft trees of a few nodes over long contexts
        {"name": "latent-long", "op": "attention", "seqs": 2, "tokens": 4, "tree": True, "ctx_min": 100003,
         "ctx_max": 131071, "heads": 16, "rank": 512, "rope": 64, "page": 64},
        # two drafted tokens a sequence in a layer with 128 heads
        {"name": "latent-128-heads", "op": "attention", "seqs": 8, "tokens": 2, "tree": False, "ctx_min": 4001,
         "ctx_max": 16411, "heads": 128, "rank": 512, "rope": 64, "page": 32},
        # draft trees of the largest pass, 64 nodes
        {"name": "latent-trees-64", "op": "attention", "seqs": 4, "tokens": 64, "tree": True, "ctx_min": 4001,
         "ctx_max": 8201, "heads": 16, "rank": 512, "rope": 64, "page": 64},
        # a small model's two layers: four branches given up and drawn anew from two sequences
        {"name": "branch-small", "op": "branch", "parents": 2, "children": 2, "layers": 2, "len_min": 100, "len_max": 500,
         "need": 8, "kind": "kv", "heads": 4, "dim": 128, "page": 64, "cache": "e4m3", "pages": 64},
        # 48 layers: eight sequences with three branches each, a part-filled page copied for every branch
        {"name": "branch-48-layers", "op": "branch", "parents": 8, "children": 3, "layers": 48, "len_min": 300, "len_max": 1100,
         "need": 16, "kind": "kv", "heads": 4, "dim": 128, "page": 64, "cache": "bf16", "pages": 300},
        # the pages of a large pool of latent rows, where the bookkeeping counts
        {"name": "branch-latent-pool", "op": "branch", "parents": 64, "children": 2, "layers": 1, "len_min": 500, "len_max": 8000,
         "need": 16, "kind": "latent", "heads": 1, "dim": 576, "page": 64, "cache": "bf16", "pages": 40000},
        # one sequence's accepted path in a small model
        {"name": "accept-small", "op": "accept", "seqs": 1, "tokens": 8, "path": 3, "layers": 2, "len_min": 100, "len_max": 200,
         "kind": "kv", "heads": 4, "dim": 128, "page": 64, "cache": "bf16", "pages": 16},
        # 16 sequences' accepted paths of 16-node trees in all 48 layers
        {"name": "accept-48-layers", "op": "accept", "seqs": 16, "tokens": 16, "path": 6, "layers": 48, "len_min": 200,
         "len_max": 900, "kind": "kv", "heads": 4, "dim": 128, "page": 16, "cache": "bf16", "pages": 1200},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "attention", "attention", "attention", "branch", "accept"))
    rank, rope = rng.choice(((512, 64), (512, 64), (256, 64), (128, 32)))
    page = rng.choice((16, 32, 64, 128))
    if op == "write":
        kind = rng.choice(("bf16", "bf16", "f32"))
        heads = rng.choice((8, 16, 20, 32))
        return {"op": op, "tokens": _log(rng, 1, 16301 if kind == "bf16" else 8150), "heads": heads, "rank": rank, "rope": rope,
                "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.6, "type": kind, "page": page, "positions": 40960}
    if op == "attention":
        heads, seqs, tokens = rng.choice((8, 12, 16, 16, 32, 64, 128)), _log(rng, 1, 64), _log(rng, 1, 64)
        # bytes as of the long contexts, products as of the largest trees
        most = min(131071, 240000 // seqs, 24_000_000 // (seqs * tokens * heads))
        if most < 1:
            seqs, most = 1, 24_000_000 // (tokens * heads)
        ctx = _log(rng, 1, most)
        return {"op": op, "seqs": seqs, "tokens": tokens, "tree": rng.random() < 0.6, "ctx_min": rng.randint(0, ctx),
                "ctx_max": ctx, "heads": heads, "rank": rank, "rope": rope, "page": page}
    layers = _log(rng, 1, 24)
    cache = rng.choice(("bf16", "bf16", "e4m3"))
    kind = rng.choice(("kv", "kv", "latent")) if cache == "bf16" else "kv"
    c = {"op": op, "layers": layers, "kind": kind, "heads": rng.choice((1, 2, 4)) if kind == "kv" else 1,
         "dim": rng.choice((64, 128)) if kind == "kv" else rank + rope, "page": page, "cache": cache}
    if op == "branch":
        c.update(parents=_log(rng, 1, 8), children=rng.randint(1, 3), need=rng.randint(1, 64))
        seqs, c["len_max"] = c["parents"] * (1 + c["children"]), rng.randint(page, 1000)
        c["len_min"] = rng.randint(1, c["len_max"])
        extra = c["need"]
    else:
        c.update(seqs=_log(rng, 1, 16), tokens=rng.randint(2, 64))
        c["path"] = rng.randint(1, c["tokens"] // 2)
        seqs, c["len_max"] = c["seqs"], rng.randint(1, 900)
        c["len_min"] = rng.randint(0, c["len_max"])
        extra = c["tokens"]
    each = -(-(c["len_max"] + extra) // page)
    c["pages"] = seqs * each + rng.randint(1, 9)
    return c


def _lens(c):
    """Cached and drafted tokens of each sequence: set by the case, not by the seed."""
    r = random.Random(c["seqs"] * 7919 + c["ctx_max"])
    ctx = [r.randint(c["ctx_min"], c["ctx_max"]) for _ in range(c["seqs"])]
    ctx[-1] = c["ctx_max"]
    n = [c["tokens"] if r.random() < 0.75 else r.randint(1, c["tokens"]) for _ in range(c["seqs"])]
    n[-1] = c["tokens"]
    return ctx, n


def _lengths(c, seqs):
    r = random.Random(seqs * 7919 + c["len_max"])
    return [r.randint(c["len_min"], c["len_max"]) for _ in range(seqs - 1)] + [c["len_max"]]


def _paths(c):
    """Accepted nodes of each sequence's tree, breadth first: the root, then nodes behind its first levels."""
    r = random.Random(c["seqs"] * 104729 + c["tokens"])
    paths = []
    for _ in range(c["seqs"]):
        k = c["path"] if not paths else r.randint(1, c["path"])
        paths.append([0] + sorted(r.sample(range(k, c["tokens"]), k - 1)))
    return paths


def _row_bytes(c):
    """Bytes of a position in all layers' caches."""
    es = _BYTES[c["cache"]]
    one = c["dim"] * es if c["kind"] == "latent" else 2 * c["heads"] * (c["dim"] * es + 4 * (c["cache"] == "e4m3"))
    return one * c["layers"]


def work(c):
    if c["op"] == "write":
        es, width = _BYTES[c["type"]], c["rank"] + c["rope"]
        b = c["tokens"] * (2 * width * es + 2 * c["heads"] * c["rope"] * es + 8 + 4 * c["rope"]) + 4 * c["rank"] * c["norm"]
        return {"bytes": b, "flops": c["tokens"] * (4 * c["rank"] * c["norm"] + 3 * c["rope"] * (c["heads"] + 1))}
    if c["op"] == "attention":
        ctx, n = _lens(c)
        width = c["rank"] + c["rope"]
        b = 2 * width * sum(x + y for x, y in zip(ctx, n)) + sum(n) * c["heads"] * (2 * width + 2 * c["rank"] + 4)
        return {"bytes": b, "flops": sum(2 * y * c["heads"] * (x + y) * (width + c["rank"]) for x, y in zip(ctx, n))}
    if c["op"] == "branch":
        lens = _lengths(c, c["parents"])
        copied = c["children"] * sum(x % c["page"] for x in lens)
        tables = (1 + 2 * c["children"]) * sum(-(-x // c["page"]) for x in lens) * 4
        return {"bytes": 2 * copied * _row_bytes(c) + tables + 4 * c["pages"], "flops": 0}
    moved = sum(i != x for p in _paths(c) for i, x in enumerate(p))
    return {"bytes": 2 * moved * _row_bytes(c) + 4 * c["pages"] + 4 * sum(map(len, _paths(c))), "flops": 0}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(c):
    """cos and sin of every position and frequency, base 10,000."""
    half = c["rope"] // 2
    w = 1e4 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(c["positions"], dtype=torch.float64, device="cuda")[:, None] * w
    return torch.stack((a.cos(), a.sin()), -1).float()


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _layers(c, g):
    """Every layer's cache in one tensor per part, [layers, pages + 1, ...] (the page behind the
    cache takes what the plain form masks out)."""
    shape = (c["layers"], c["pages"] + 1, c["page"])
    if c["kind"] == "latent":
        return {"rows": torch.randn((*shape, c["dim"]), generator=g, device="cuda", dtype=torch.bfloat16)}
    kv = lambda: torch.randn((*shape, c["heads"], c["dim"]), generator=g, device="cuda", dtype=torch.bfloat16)
    if c["cache"] == "bf16":
        return {"k": kv(), "v": kv()}
    # codes of N(0, 1) rows whose largest magnitudes lie near 448
    codes = lambda: kv().mul_(130).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = lambda: torch.rand((*shape[:2], c["heads"], c["page"]), generator=g, device="cuda").mul_(0.004).add_(0.006)
    return {"k": codes(), "v": codes(), "k_scale": scales(), "v_scale": scales()}


def prepare(case, seed):
    g, rng, c = _generator(seed), np.random.default_rng(seed), case
    s = {"case": c, "op": c["op"]}
    if c["op"] == "write":
        t = _TYPES[c["type"]]
        # latents and rotary keys are two parts of one projection's output; the rotary channels of
        # the queries are a part of theirs
        both = torch.randn((c["tokens"], c["rank"] + c["rope"]), generator=g, device="cuda", dtype=t)
        s["latent"], s["k"] = both.split([c["rank"], c["rope"]], 1)
        s["q"] = torch.randn((c["tokens"], c["heads"], 128 + c["rope"]), generator=g, device="cuda", dtype=t)[..., 128:]
        s["norm"] = torch.rand(c["rank"], generator=g, device="cuda").add_(0.5) if c["norm"] else None
        start = int(rng.integers(0, c["positions"] - c["tokens"] + 1))
        s["positions"] = torch.arange(start, start + c["tokens"], dtype=torch.int32, device="cuda")
        s["table"] = _table(c)
        pages = -(-c["tokens"] // c["page"]) + 3
        order = torch.from_numpy(rng.permutation(pages)).cuda()
        i = torch.arange(c["tokens"], device="cuda")
        slots = order[i // c["page"]] * c["page"] + i % c["page"]
        if c["tokens"] > 4:   # the padding of a batch's last rows
            slots[-2:] = -1
        s["slots"] = slots.int()
        s["rows"] = torch.randn((pages + 1, c["page"], c["rank"] + c["rope"]), generator=g, device="cuda", dtype=t)
    elif c["op"] == "attention":
        ctx, n = _lens(c)
        need = [-(-(a + b) // c["page"]) for a, b in zip(ctx, n)]
        pages = sum(need) + 3
        order, at = rng.permutation(pages).astype(np.int32), 0
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
        s["ctx"], s["starts"] = _int(ctx), _int(np.concatenate([[0], np.cumsum(n)]).tolist())
        s["rows"] = torch.randn((pages, c["page"], c["rank"] + c["rope"]), generator=g, device="cuda", dtype=torch.bfloat16)
        # queries whose scores spread over several units, so that some positions stand out
        s["q"] = torch.randn((sum(n), c["heads"], c["rank"] + c["rope"]), generator=g, device="cuda", dtype=torch.bfloat16)
        s["scale"] = 2.5 / math.sqrt(c["rank"] + c["rope"])
    else:
        s["parts"] = _layers(c, g)
        branch = c["op"] == "branch"
        owners = c["parents"] if branch else c["seqs"]
        seqs = owners * (1 + c["children"]) if branch else owners
        lens = _lengths(c, owners)
        need = c["need"] if branch else c["tokens"]
        width = -(-(c["len_max"] + need) // c["page"]) + 1
        order, at = rng.permutation(c["pages"]).astype(np.int32), 0
        table, refs = np.zeros((seqs, width), np.int32), np.zeros(c["pages"], np.int32)
        held, length = np.zeros(seqs, np.int32), np.zeros(seqs, np.int32)
        for b, x in enumerate(lens):
            held[b], length[b] = -(-x // c["page"]), x
            table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
            refs[table[b, :held[b]]] += 1
        if branch:   # the branches hold what an earlier step gave them: their parents' full pages
            s["src"] = _int([b for b in range(owners) for _ in range(c["children"])])
            s["dst"] = _int(list(range(owners, seqs)))
            for d, b in zip(range(owners, seqs), s["src"].tolist()):
                held[d], length[d] = lens[b] // c["page"], lens[b] // c["page"] * c["page"]
                table[d, :held[d]] = table[b, :held[d]]
                refs[table[d, :held[d]]] += 1
        else:
            paths = _paths(c)
            s["path"] = _int([p + [0] * (c["path"] - len(p)) for p in paths])
            s["count"] = _int([len(p) for p in paths])
            s["after"] = _int([0] * seqs)
        s["need"] = _int([0 if branch and b < owners else need for b in range(seqs)])   # the branches grow
        s.update(refs=_int(refs.tolist()), table=_int(table.tolist()), held=_int(held.tolist()), length=_int(length.tolist()),
                 got=_int([0] * seqs))
    if own:
        from moe_speculative_decoding_gb300 import api
        if c["op"] in ("write", "attention"):
            s["cache"] = api.LatentCache(s["rows"][:pages], c["rank"])
            if c["op"] == "attention":
                s["ws"] = api.latent_attention_workspace(s["cache"], s["q"].shape[0], c["seqs"], c["heads"])
        else:
            x, n = s["parts"], c["pages"]
            caches = [api.LatentCache(x["rows"][i, :n], c["dim"] - 64 if c["dim"] > 160 else c["dim"] - 32) if "rows" in x else
                      api.KVCache(*(x[p][i, :n] if p in x else None for p in ("k", "v", "k_scale", "v_scale")))
                      for i in range(c["layers"])]
            s["pool"] = api.PagePool(caches, s["refs"], s["table"], s["held"])
    return s


# ---------------------------------------------------------------- the library's calls

def _call(s):
    from moe_speculative_decoding_gb300 import api
    c = s["case"]
    if s["op"] == "write":
        q = api.latent_write(s["cache"], s["latent"], s["k"], s["slots"], norm=s["norm"], eps=_EPS, q=s["q"],
                             positions=s["positions"], table=s["table"], interleaved=c["interleaved"])
        return s["rows"][:-1], q
    if s["op"] == "attention":
        return api.latent_attention(s["cache"], s["q"], s["starts"], s["ctx"], s["page_table"], s["scale"], mask=s["mask"],
                                    max_tokens=c["tokens"], return_lse=True, ws=s["ws"])
    pool = s["pool"]
    if s["op"] == "branch":
        api.pages_free(pool, s["dst"], s["length"])
        api.pages_fork(pool, s["src"], s["dst"], s["length"])
        api.pages_reserve(pool, s["length"], s["need"], got=s["got"])
        return _paged(s)
    api.pages_reserve(pool, s["length"], s["need"], got=s["got"])
    api.pages_accept(pool, s["length"], s["path"], s["count"], after=s["after"])
    return _paged(s) + [s["after"]]


def _paged(s):
    """The pool and every layer's cache: codes as the 8-bit floats they are."""
    seen = [s[x] for x in ("refs", "table", "held", "length", "got")]
    return seen + [x[:, :-1].view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x[:, :-1] for x in s["parts"].values()]


# ---------------------------------------------------------------- plain forms

def _rotate(x, s):
    """[tokens, heads, rope] in fp32."""
    x, t = x.float(), s["table"][s["positions"].long()][:, None]
    cos, sin = t[..., 0], t[..., 1]
    if s["case"]["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _write(s):
    c, y = s["case"], s["latent"].float()
    if s["norm"] is not None:
        y = y * (y.square().mean(-1, keepdim=True) + _EPS).rsqrt() * s["norm"]
    row = torch.cat((y, _rotate(s["k"][:, None], s)[:, 0]), -1)
    slots = s["slots"].long()
    slots = torch.where(slots < 0, (s["rows"].shape[0] - 1) * c["page"], slots)   # the page beyond the cache
    s["rows"][slots // c["page"], slots % c["page"]] = row.to(s["rows"].dtype)
    return s["rows"][:-1], _rotate(s["q"], s).to(s["q"].dtype)


def _attend(s):
    c, q, starts, ctx = s["case"], s["q"], s["starts"].long(), s["ctx"].long()
    total, seqs, n, h = q.shape[0], c["seqs"], c["tokens"], c["heads"]
    token = torch.arange(total, device=q.device)
    b = torch.searchsorted(starts, token, right=True) - 1
    i = token - starts[b]
    pick = (starts[:-1, None] + torch.arange(n, device=q.device)).clamp(max=total - 1)
    rows = s["rows"][s["page_table"].long()].flatten(1, 2).float()
    scores = q[pick].float().flatten(1, 2) @ rows.transpose(1, 2) * s["scale"]
    drafted = torch.arange(rows.shape[1], device=q.device) - ctx[:, None]
    if s["mask"] is None:
        seen = drafted[:, None] <= torch.arange(n, device=q.device)[:, None]
    else:
        seen = (s["mask"][pick][..., None] >> drafted.clamp(0, 63)[:, None] & 1 > 0) | (drafted[:, None] < 0)
    seen = seen & (drafted < (starts[1:] - starts[:-1])[:, None])[:, None]
    scores = scores.view(seqs, n, h, -1).masked_fill(~seen[:, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (scores - top).exp()
    z = e.sum(-1, keepdim=True)
    out = (e.flatten(1, 2) @ rows[..., :c["rank"]]).view(seqs, n, h, -1) / torch.where(z > 0, z, torch.ones_like(z))
    return out[b, i].to(q.dtype), (z.log() + top)[..., 0][b, i]


def _free(s, ids):
    refs, table, held = s["refs"], s["table"], s["held"]
    j = torch.arange(table.shape[1], device=refs.device)
    mine = j < held[ids][:, None]
    refs.index_add_(0, table[ids].flatten(), -mine.flatten().int())
    held[ids] = 0
    s["length"][ids] = 0


def _fork(s, src, dst):
    refs, table, held = s["refs"], s["table"], s["held"]
    k = -(-s["length"][src] // s["case"]["page"])
    mine = torch.arange(table.shape[1], device=refs.device) < k[:, None]
    table[dst] = torch.where(mine, table[src], table[dst])
    refs.index_add_(0, table[src].flatten(), mine.flatten().int())
    held[dst] = k
    s["length"][dst] = s["length"][src]


def _reserve(s):
    refs, table, held, length, need, page = s["refs"], s["table"], s["held"], s["length"], s["need"], s["case"]["page"]
    seqs, j = table.shape[0], torch.arange(table.shape[1], device=refs.device)
    first = length // page
    at = table.gather(1, first[:, None].long())[:, 0]
    shared = (length % page > 0) & (need > 0) & (refs[at] > 1)
    same = (at[:, None] == at) & shared[:, None] & shared
    before = same.tril(-1).sum(1)   # holders before this one that take a copy
    copy = shared & (refs[at] - before > 1)
    want = torch.maximum(held, torch.where(need > 0, -(-(length + need) // page), 0))
    extra = want - held + copy
    upto = extra.cumsum(0)
    free = refs == 0
    order = torch.argsort((~free).int(), stable=True)
    ok = (extra == 0) | (upto <= free.sum())
    # from the first that fails on, only those before it have given shared pages up
    served = (~ok).cumsum(0) == 0
    ok &= ~(shared & (refs[at] - (same.tril(-1) & served).sum(1) > 1) & ~served)
    copy = copy & ok
    at_new = (upto - extra).long()
    # the copy takes the first page, the pages behind those held the others
    new = order[at_new.clamp(max=refs.shape[0] - 1)].int()
    refs.index_add_(0, at, -copy.int())
    refs.index_add_(0, new, copy.int())
    place = (at_new + copy)[:, None] + j - held[:, None]
    fresh = (j >= held[:, None]) & (j < want[:, None]) & ok[:, None]
    pages = order[place.clamp(0, refs.shape[0] - 1)].int()
    refs.index_add_(0, pages.flatten(), fresh.flatten().int())
    table.copy_(torch.where(fresh, pages, table))
    table.scatter_(1, first[:, None].long(), torch.where(copy, new, table.gather(1, first[:, None].long())[:, 0])[:, None])
    held.copy_(torch.where(ok, want, held))
    s["got"].copy_(ok)
    # rows below the length, in all layers; the page behind the cache takes the rest
    r = torch.arange(page, device=refs.device)
    keep = copy[:, None] & (r < (length % page)[:, None])
    target = torch.where(keep, new[:, None], s["case"]["pages"]).long()
    for name, x in s["parts"].items():
        a = at[:, None].long().expand(seqs, page)
        if name.endswith("scale"):
            x[:, target, :, r] = x[:, a, :, r]
        else:
            x[:, target, r] = x[:, a, r]


def _accept(s):
    refs, table, held, ctx, page = s["refs"], s["table"], s["held"], s["length"], s["case"]["page"]
    path, count = s["path"].long(), s["count"].long()
    i = torch.arange(path.shape[1], device=refs.device)
    old, new = ctx[:, None] + path, (ctx[:, None] + i).expand_as(path)
    keep = i < count[:, None]
    where = lambda p: table.gather(1, (p // page).clamp(max=table.shape[1] - 1)).long()
    source, target = where(old), torch.where(keep, where(new), s["case"]["pages"])
    for name, x in s["parts"].items():   # read before they are written
        if name.endswith("scale"):
            x[:, target, :, new % page] = x[:, source, :, old % page]
        else:
            x[:, target, new % page] = x[:, source, old % page]
    s["after"].copy_(ctx + count)
    left = -(-s["after"] // page)
    j = torch.arange(table.shape[1], device=refs.device)
    refs.index_add_(0, table.flatten(), -((j >= left[:, None]) & (j < held[:, None])).flatten().int())
    held.copy_(torch.minimum(held, left))


def run(s):
    if own:
        return _call(s)
    if s["op"] == "write":
        return _write(s)
    if s["op"] == "attention":
        return _attend(s)
    if s["op"] == "branch":
        _free(s, s["dst"])
        _fork(s, s["src"], s["dst"])
        _reserve(s)
        return _paged(s)
    _reserve(s)
    _accept(s)
    return _paged(s) + [s["after"]]


# ---------------------------------------------------------------- in 64 bits

def _turned(x, s):
    """Rotation as the product of each pair, taken as a complex number, with e^(i angle)."""
    x = x.double()
    t = s["table"].double()[s["positions"].long()]
    turn = torch.complex(t[..., 0], t[..., 1])[:, None]
    half = x.shape[-1] // 2
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(x.reshape(*x.shape[:2], half, 2).contiguous()) * turn
        return torch.view_as_real(z).reshape(x.shape)
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
    return torch.cat((z.real, z.imag), -1)


def _pages_by_hand(s):
    """The steps on lists, one sequence after the other: the pool after them, and the rows of one
    place (page, row) that come from another."""
    c = s["case"]
    page, refs, table, held, length = c["page"], *(s[x].tolist() for x in ("refs", "table", "held", "length"))
    need, got, moved = s["need"].tolist(), [], {}
    if c["op"] == "branch":
        for d in s["dst"].tolist():
            for p in table[d][:held[d]]:
                refs[p] -= 1
            held[d] = 0
        for a, d in zip(s["src"].tolist(), s["dst"].tolist()):
            held[d], length[d] = math.ceil(length[a] / page), length[a]
            for k in range(held[d]):
                table[d][k] = table[a][k]
                refs[table[d][k]] += 1
    free, out = [p for p, r in enumerate(refs) if r == 0], False   # the free pages as the call finds them
    for b in range(len(held)):
        k = length[b] // page
        copy = need[b] > 0 and length[b] % page > 0 and refs[table[b][k]] > 1
        want = max(held[b], math.ceil((length[b] + need[b]) / page)) if need[b] > 0 else held[b]
        extra = want - held[b] + copy
        out = out or extra > len(free)
        got.append(int(extra == 0 or not out))
        if not got[b]:
            continue
        if copy:
            old, table[b][k] = table[b][k], free.pop(0)
            refs[old] -= 1
            refs[table[b][k]] += 1
            moved.update({(table[b][k], r): (old, r) for r in range(length[b] % page)})
        for k in range(held[b], want):
            table[b][k] = free.pop(0)
            refs[table[b][k]] += 1
        held[b] = want
    after = None
    if c["op"] == "accept":
        after = []
        for b, (path, n) in enumerate(zip(s["path"].tolist(), s["count"].tolist())):
            spot = lambda x: (table[b][x // page], x % page)
            moved.update({spot(length[b] + i): spot(length[b] + path[i]) for i in range(n)})
            after.append(length[b] + n)
            while held[b] > math.ceil(after[b] / page):
                held[b] -= 1
                refs[table[b][held[b]]] -= 1
    return [refs, table, held, length, got], moved, after


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "write":
        x = s["latent"].double()
        if s["norm"] is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["rank"] + _EPS) * s["norm"].double()
        where = s["slots"].long()
        keep = where >= 0
        rows = s["rows"][:-1].double()
        rows[where[keep] // c["page"], where[keep] % c["page"]] = torch.cat((x, _turned(s["k"][:, None], s)[:, 0]), -1)[keep]
        return rows, _turned(s["q"], s)
    if c["op"] in ("branch", "accept"):
        lists, moved, after = _pages_by_hand(s)
        parts = []
        to, of = (torch.tensor(x, dtype=torch.long, device="cuda").view(-1, 2).T for x in (list(moved), list(moved.values())))
        for name, x in s["parts"].items():
            x = x[:, :-1].view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x[:, :-1]
            y = x.double()
            if name.endswith("scale"):
                y[:, to[0], :, to[1]] = x[:, of[0], :, of[1]].double()
            else:
                y[:, to[0], to[1]] = x.view(torch.uint8)[:, of[0], of[1]].view(x.dtype).double()
            parts.append(y)
        return [_int(x) for x in lists] + parts + ([_int(after)] if after is not None else [])
    if work(c)["flops"] > 2e11:
        return None
    outs, lses, starts, ctx = [], [], s["starts"].tolist(), s["ctx"].tolist()
    masks = s["mask"].tolist() if s["mask"] is not None else None
    for b in range(c["seqs"]):
        n = starts[b + 1] - starts[b]
        x = s["rows"][s["page_table"][b, :-(-(ctx[b] + n) // c["page"])].long()].flatten(0, 1)[:ctx[b] + n].double()
        see = np.ones((n, ctx[b] + n), bool)
        for i in range(n):
            for j in range(n):
                see[i, ctx[b] + j] = j <= i if masks is None else (masks[starts[b] + i] >> j) & 1
        a = torch.einsum("nhc,pc->hnp", s["q"][starts[b]:starts[b + 1]].double(), x) * s["scale"]
        a = a.masked_fill(~torch.from_numpy(see).cuda(), -math.inf)
        lses.append(torch.logsumexp(a, -1).T)
        outs.append(torch.einsum("hnp,pc->nhc", torch.softmax(a, -1), x[:, :c["rank"]]))
    return torch.cat(outs), torch.cat(lses)

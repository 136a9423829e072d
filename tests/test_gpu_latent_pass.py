"""Latent rows, attention over them and the pages under them as they are used together: sequences that
branch from one another, and the example's speculative rounds."""
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

from latent_util import LatentPass
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("heads,rank,rope,page", [(16, 512, 64, 16), (5, 128, 32, 8), (8, 256, 64, 64)])
def test_branches_see_their_own_rows(heads, rank, rope, page):
    """Prompts, branches that share their pages, and different tokens behind them: every sequence's output is
    that of attention over its own tokens, in both layers, whatever pages they lie in."""
    rng, g = random.Random(page), torch.Generator().manual_seed(page)
    seqs, layers, width = 6, 2, rank + rope
    caches = [api.latent_cache(70, page, rank, rope) for _ in range(layers)]
    pool = api.page_pool(caches, seqs, 1 + 160 // page)
    ws = api.latent_attention_workspace(caches[0], 64, seqs, heads)
    rows = [[torch.zeros((0, width), dtype=BF16) for _ in range(seqs)] for _ in range(layers)]   # what they hold

    def step(active, n):
        """n[b] drafted tokens for every active sequence; of their tree a random path is accepted."""
        length = [len(rows[0][b]) for b in range(seqs)]
        need = [n[b] if b in active else 0 for b in range(seqs)]
        assert api.pages_reserve(pool, i32(length), i32(need)).tolist() == [1] * seqs
        owner = [b for b in active for _ in range(n[b])]
        at = [length[b] + i for b in active for i in range(n[b])]
        table = pool.table.tolist()
        slots = i32([table[b][p // page] * page + p % page for b, p in zip(owner, at)])
        masks = []
        for b in active:
            seen = []
            for i in range(n[b]):
                parent = rng.randrange(-1, i) if i else -1
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
            masks += seen
        for layer in range(layers):
            new = torch.randn((len(owner), width), generator=g).to(BF16)
            q = torch.randn((len(owner), heads, width), generator=g).to(BF16)
            dev = new.cuda()
            api.latent_write(caches[layer], dev[:, :rank], dev[:, rank:], slots)
            p = LatentPass.__new__(LatentPass)
            p.__dict__.update(ctx=[length[b] for b in active], n=[n[b] for b in active], heads=heads, rank=rank, rope=rope, page=page,
                              starts=np.cumsum([0] + [n[b] for b in active]), mask=np.array(masks, np.uint64), q=q,
                              rows=torch.zeros((1, page, width), dtype=BF16), scale=width ** -0.5)
            held = [torch.cat((rows[layer][b], new[[i for i, o in enumerate(owner) if o == b]])) for b in active]
            p.cached = lambda i: held[i].double()
            out, lse = api.latent_attention(caches[layer], q.cuda(), i32(p.starts.tolist()), i32(p.ctx), pool.table[active].contiguous(),
                                            p.scale, mask=torch.from_numpy(p.mask.view(np.int64)).cuda(), max_tokens=max(p.n),
                                            return_lse=True, ws=ws)
            p.check(api, out, lse)
            for b, x in zip(active, held):
                rows[layer][b] = x
        path, count = [[0] * max(n) for _ in range(seqs)], [-1] * seqs
        for b in active:
            keep = sorted(rng.sample(range(n[b]), rng.randint(1, n[b])))
            path[b][:len(keep)], count[b] = keep, len(keep)
            for layer in range(layers):
                x = rows[layer][b]
                rows[layer][b] = torch.cat((x[:length[b]], x[length[b]:][keep]))
        after = api.pages_accept(pool, i32(length), i32(path), i32(count))
        assert after.tolist() == [len(rows[0][b]) for b in range(seqs)]

    step([0, 1], [40, 33, 0, 0, 0, 0])
    step([0, 1], [9, 17, 0, 0, 0, 0])
    for _ in range(3):
        length = i32([len(rows[0][b]) for b in range(seqs)])
        api.pages_fork(pool, i32([0, 0, 1, 0]), i32([2, 3, 4, 5]), length)
        for layer in range(layers):
            for d, s in ((2, 0), (3, 0), (4, 1), (5, 0)):
                rows[layer][d] = rows[layer][s]
        step([2, 3, 4], [0, 0, 5, 1, 7, 0])       # the branches write, their parents do not
        step([0, 1, 2, 3, 4, 5], [3, 2, 4, 4, 1, 6])
        api.pages_free(pool, i32([2, 3, 4, 5, 2]))
        for layer in range(layers):
            for d in (2, 3, 4, 5):
                rows[layer][d] = rows[layer][d][:0]
    assert api.last_device_error(ws) == 0 and api.last_device_error(pool.ws) == 0
    api.pages_free(pool, i32([0, 1]))
    assert pool.refs.eq(0).all() and pool.held.eq(0).all()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "verify_pass.py")
    spec = importlib.util.spec_from_file_location("verify_pass", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_rounds_of_latent_layers_agree_with_a_prefill(example):
    """As for layers with key heads: the logits that follow the last accepted token against those of a fresh
    prefill, by direction (16 bits in and between the layers may swap an expert)."""
    prompts = torch.randint(example.VOCAB, (3, 70), generator=torch.Generator().manual_seed(2)).cuda()
    plain, _ = example.decode(example.Model(3, attention="latent"), prompts, 8, seed=3)

    def guess(trees, tokens):
        for b, t in enumerate(tokens):
            rest = plain[b][len(t) - 70:]
            for node, k in ((1, 0), (3, 1), (6, 2)):   # the root's child, its second child, that one's first
                if k < len(rest):
                    trees[b, node] = rest[k]

    model = example.Model(3, attention="latent")
    example.model_guess = guess
    try:
        out, logits = example.decode(model, prompts, 3, seed=4)
    finally:
        example.model_guess = None
    assert all(api.last_device_error(ws) == 0 for ws in (model.attn_ws, model.ws, model.pool.ws))
    assert max(len(o) for o in out) > 4   # paths longer than a node
    assert model.pool.held.tolist() == [-(-(69 + len(o)) // example.PAGE) for o in out]
    assert model.pool.refs.sum().item() == model.pool.held.sum().item()
    for b in range(3):
        seen = torch.cat([prompts[b], torch.tensor(out[b][:-1], device="cuda")])[None]
        ref = example.prefill(example.Model(1, attention="latent"), seen)[0]
        near = torch.nn.functional.cosine_similarity(logits, ref[None], dim=1)
        assert near[b].item() > 0.98
        assert max(near[i].item() for i in range(3) if i != b) < 0.9   # the other sequences'

"""Speculative decoding with draft trees on one GPU: every pass writes its keys and values into a paged
cache, attends over it, routes and runs the experts, all through the public calls.

    python examples/verify_pass.py [--cache bf16|e4m3] [--rounds 4]

The model is random (two layers of the 128-expert shape), and so are the drafts: what is shown is the
order of calls.  A round drafts a tree for each sequence, verifies all trees in one pass, follows each
tree's longest path of greedy tokens, and moves that path's rows to where the next pass expects them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_speculative_decoding_gb300 import api, synth
from moe_speculative_decoding_gb300.configs import QWEN3

HEADS, KV_HEADS, DIM, PAGE, PAGES_EACH, VOCAB = 32, 4, 128, 64, 8, 1024
# a draft tree: each node's parent (-1: the last accepted token), parents first
PARENTS = [-1, 0, 0, 1, 1, 2, 3]


class Rotary(torch.autograd.Function):
    """Rotation with its gradient: the transpose of a rotation is the rotation back."""

    @staticmethod
    def forward(ctx, x, positions, table):
        ctx.save_for_backward(positions, table)
        return api.rope(x.contiguous(), None, positions, table)[0]

    @staticmethod
    def backward(ctx, g):
        positions, table = ctx.saved_tensors
        return api.rope(g.contiguous(), None, positions, table, inverse=True)[0], None, None


class Model:
    def __init__(self, seqs, layers=2, cache="bf16", seed=0):
        wl, g = QWEN3, torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16()
        self.embed = 0.1 * torch.randn(VOCAB, wl.d, generator=g, device="cuda").bfloat16()   # so that the layers have a say
        self.head = torch.randn(VOCAB, wl.d, generator=g, device="cuda")
        self.proj = [(rand(wl.d, HEADS * DIM), rand(wl.d, KV_HEADS * DIM), rand(wl.d, KV_HEADS * DIM), rand(HEADS * DIM, wl.d),
                      rand(wl.d, wl.N).float()) for _ in range(layers)]
        self.layer = api.make_layer(wl.d, wl.f, wl.N, wl.m)
        self.experts = [synth.expert_weights(wl.N, wl.f, wl.d, torch.bfloat16, seed + i, device="cuda") for i in range(layers)]
        self.caches = [api.kv_cache(seqs * PAGES_EACH, PAGE, KV_HEADS, DIM, cache) for _ in range(layers)]
        self.pages = torch.randperm(seqs * PAGES_EACH, generator=torch.Generator().manual_seed(seed)).int().view(seqs, -1).cuda()
        self.rope = api.rope_table(PAGES_EACH * PAGE, *api.rope_frequencies(DIM))
        # workspaces live as long as the model
        self.ws = api.workspace(self.layer, 64)
        self.attn_ws = api.tree_attention_workspace(self.caches[0], 64, seqs, HEADS)

    def slots(self, seq, at):
        """Cache slots of places `at` of sequences `seq` (both int64)."""
        return self.pages[seq, at // PAGE] * PAGE + (at % PAGE).int()

    def run(self, tokens, seq, at, positions, starts, lengths, mask=None):
        """One pass of up to 64 tokens: logits.  seq, at: each token's sequence and place in the cache;
        starts: the sequences' bounds among the tokens; lengths: what the cache holds before them."""
        slots, h = self.slots(seq, at), self.embed[tokens]
        for (wq, wk, wv, wo, router), experts, cache in zip(self.proj, self.experts, self.caches):
            x = torch.nn.functional.rms_norm(h, h.shape[1:])
            q, k, v = ((x @ w).view(-1, w.shape[1] // DIM, DIM) for w in (wq, wk, wv))
            q = api.kv_write(cache, k, v, slots, q=q, positions=positions, table=self.rope, ws=self.attn_ws)
            o = api.tree_attention(cache, q, starts, lengths, self.pages, mask=mask, ws=self.attn_ws)
            h = h + o.view(len(tokens), -1) @ wo
            x = torch.nn.functional.rms_norm(h, h.shape[1:])
            ids, gates = api.route_topm(x.float() @ router, self.layer.m)
            h = h + api.expert_op_dedup_ids(self.layer, experts, x, ids, gates, ws=self.ws).to(h.dtype)
        return torch.nn.functional.rms_norm(h, h.shape[1:]).float() @ self.head.T

    def move(self, seq, source, target):
        """Rows of places `source` of the cache to `target` (read before they are written)."""
        old, new = self.slots(seq, source), self.slots(seq, target)
        for cache in self.caches:
            k, v = api.kv_read(cache, old, dtype=torch.float32)
            api.kv_write(cache, k, v, new)


def check_room(tokens):
    """Places beyond a sequence's pages have no slot (and an index on the device is not checked on the host)."""
    if tokens > PAGES_EACH * PAGE:
        raise ValueError(f"a sequence would need {tokens} places of the cache and has {PAGES_EACH * PAGE}")


def prefill(model, prompts):
    """The prompts [seqs, n] as chains, a pass of up to 64 tokens at a time; the last token's logits."""
    seqs, n = prompts.shape
    check_room(n)
    step = max(1, 64 // seqs)
    for i in range(0, n, step):
        m = min(step, n - i)
        seq = torch.arange(seqs, device="cuda").repeat_interleave(m)
        at = torch.arange(i, i + m, device="cuda").repeat(seqs)
        logits = model.run(prompts[:, i:i + m].reshape(-1), seq, at, at.int(),
                           torch.arange(0, seqs * m + 1, m, dtype=torch.int32, device="cuda"),
                           torch.full((seqs,), i, dtype=torch.int32, device="cuda"))
    return logits.view(seqs, m, -1)[:, -1]


def decode(model, prompts, rounds, seed=0):
    """Greedy speculative decoding.  Returns each sequence's tokens after the prompt and the logits that
    follow its last one."""
    g = torch.Generator().manual_seed(seed)
    seqs, n = prompts.shape
    T = len(PARENTS) + 1   # a pass's tokens of a sequence: its last token, which no pass has seen, and the tree
    parents = [-1] + [p + 1 for p in PARENTS]
    depth, words = [0] * T, [1] + [0] * (T - 1)
    for i in range(1, T):
        depth[i], words[i] = depth[parents[i]] + 1, words[parents[i]] | 1 << i
    mask = torch.tensor(words * seqs, device="cuda")
    seq = torch.arange(seqs, device="cuda").repeat_interleave(T)
    starts = torch.arange(0, seqs * T + 1, T, dtype=torch.int32, device="cuda")
    logits = prefill(model, prompts)
    last, length = logits.argmax(-1).tolist(), [n] * seqs
    out, final = [[t] for t in last], [logits[b] for b in range(seqs)]
    for _ in range(rounds):
        check_room(max(length) + T)
        # a drafter would propose likely tokens; these are random
        trees = torch.randint(VOCAB, (seqs, T), generator=g)
        trees[:, 0] = torch.tensor(last)
        if model_guess is not None:
            model_guess(trees, [prompts[b].tolist() + out[b] for b in range(seqs)])
        lengths = torch.tensor(length, dtype=torch.int32, device="cuda")
        at = lengths.long()[seq] + torch.arange(T, device="cuda").repeat(seqs)
        positions = lengths[seq] + torch.tensor(depth * seqs, dtype=torch.int32, device="cuda")
        logits = model.run(trees.view(-1).cuda(), seq, at, positions, starts, lengths, mask).view(seqs, T, -1)
        best = logits.argmax(-1).tolist()
        who, source, target = [], [], []
        for b in range(seqs):
            path = [0]
            while (child := next((i for i in range(1, T) if parents[i] == path[-1] and int(trees[b, i]) == best[b][path[-1]]), None)):
                path.append(child)
            for d, i in enumerate(path):
                if i != d:   # the path's rows become consecutive
                    who.append(b)
                    source.append(length[b] + i)
                    target.append(length[b] + d)
            out[b] += [int(trees[b, i]) for i in path[1:]] + [best[b][path[-1]]]
            length[b] += len(path)
            last[b], final[b] = out[b][-1], logits[b, path[-1]]
        if who:
            model.move(*(torch.tensor(x, device="cuda") for x in (who, source, target)))
    return out, torch.stack(final)


model_guess = None   # fills a round's trees from the tokens so far; the tests set it


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--cache", default="bf16", choices=("bf16", "e4m3"))
    ap.add_argument("--rounds", type=int, default=4)
    a = ap.parse_args()
    prompts = torch.randint(VOCAB, (4, 100), generator=torch.Generator().manual_seed(1)).cuda()
    model = Model(4, cache=a.cache)
    out, _ = decode(model, prompts, a.rounds)
    for b, tokens in enumerate(out):
        print(f"sequence {b}: {len(tokens)} tokens in {a.rounds + 1} passes: {tokens}")
    print("device errors:", api.last_device_error(model.attn_ws), api.last_device_error(model.ws))
    x = torch.randn(16, HEADS, DIM, device="cuda", requires_grad=True)
    positions = torch.arange(16, dtype=torch.int32, device="cuda")
    Rotary.apply(x, positions, model.rope).square().sum().backward()   # a rotation keeps lengths: the gradient is 2 x
    print("rotation's gradient, largest error: %.1e" % (x.grad - 2 * x.detach()).abs().max().item())


if __name__ == "__main__":
    main()

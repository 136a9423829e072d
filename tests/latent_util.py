"""64-bit references and error bounds of latent attention and of the pages of a cache, written from the
formulas on the CPU."""
import math

import numpy as np
import torch


class LatentPass:
    """A seeded batch for latent attention: ragged contexts and draft trees over shuffled pages."""

    def __init__(self, ctx, n, heads, rank, rope, page, kind=torch.bfloat16, q_kind=None, tree=True, seed=0, spread=2.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.n, self.heads, self.rank, self.rope, self.page = list(ctx), list(n), heads, rank, rope, page
        need = [max(1, -(-(a + b) // page)) for a, b in zip(ctx, n)]
        pages = sum(need) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.zeros((len(ctx), max(need) + 1), np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.mask = None
        if tree:
            words = []
            for k in n:
                seen = []
                for i in range(k):
                    parent = int(rng.integers(-1, i)) if i else -1
                    seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
                words += seen
            self.mask = np.array(words, np.uint64)
        self.q = (torch.randn((sum(n), heads, rank + rope), generator=g) * spread).to(q_kind or kind)
        self.rows = torch.randn((pages, page, rank + rope), generator=g).to(kind)
        self.scale = (rank + rope) ** -0.5

    def cached(self, b):
        """[ctx + n, rank + rope] of one sequence."""
        p = np.arange(self.ctx[b] + self.n[b])
        return self.rows[torch.from_numpy(self.table[b][p // self.page].astype(np.int64)), torch.from_numpy(p % self.page)].double()

    def at(self, b, p):
        """The place (page, row) of position p of sequence b."""
        return int(self.table[b][p // self.page]), p % self.page

    def sees(self, b):
        length, n = self.ctx[b] + self.n[b], self.n[b]
        see = torch.ones((n, length), dtype=torch.bool)
        for i in range(n):
            bits = (1 << (i + 1)) - 1 if self.mask is None else int(self.mask[self.starts[b] + i])
            for j in range(n):
                see[i, self.ctx[b] + j] = bool((bits >> j) & 1)
        return see

    def reference(self, p_eps, out_bf16):
        """(out, lse, out bound, lse bound) in float64.  A score of w = rank + rope products, each 2^-24 off
        and summed in any order in fp32, is off by at most ds = (w + 4) 2^-24 scale sum |q||k|, so a weight by 2 ds
        relative; exponential, sums of positive terms in tiles and the division add at most 2^-18; p_eps
        is the rounding of the weights for the product with the latents.  All of that scales
        sum p |c|; rounding the result to bf16 adds 2^-8 |out|."""
        total, w = self.q.shape[0], self.rank + self.rope
        out = torch.zeros((total, self.heads, self.rank), dtype=torch.float64)
        lse = torch.full((total, self.heads), -math.inf, dtype=torch.float64)
        ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
        for b in range(len(self.n)):
            see, x = self.sees(b), self.cached(b)
            x0 = torch.where(see.any(0)[:, None], x, torch.zeros_like(x))
            for i in range(self.n[b]):
                t, seen = int(self.starts[b]) + i, see[i]
                if not bool(seen.any()):
                    continue
                q, k = self.q[t].double(), x[seen]
                s = q @ k.T * self.scale
                ds = (w + 4) * 2.0 ** -24 * self.scale * (q.abs() @ x0[seen].abs().T).amax(-1)
                top = s.amax(-1)
                e = torch.exp(s - top[:, None])
                z = e.sum(-1)
                p = e / z[:, None]
                out[t] = p @ k[:, :self.rank]
                ob[t] = (p_eps + 2 * ds + 2.0 ** -18)[:, None] * (p @ k[:, :self.rank].abs())
                lse[t] = torch.log(z) + top
                lb[t] = ds + 2.0 ** -20 * (1 + top.abs())
        if out_bf16:
            ob = ob + 2.0 ** -8 * (out.abs() + ob)
        return out, lse, ob, lb

    def device(self, api, dev="cuda"):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        return dict(cache=api.LatentCache(self.rows.to(dev), self.rank), q=self.q.to(dev), q_start=t(self.starts),
                    ctx=t(np.array(self.ctx, np.int32)), page_table=t(self.table), scale=self.scale,
                    mask=None if self.mask is None else t(self.mask.view(np.int64)))

    def on_tensor_cores(self):
        return self.q.dtype == torch.bfloat16 and self.rows.dtype == torch.bfloat16 and self.rope <= 64 and self.page % 8 == 0

    def check(self, api, out, lse):
        ref, ref_lse, bound, lse_bound = self.reference(2.0 ** -8 if self.on_tensor_cores() else 0.0, self.q.dtype == torch.bfloat16)
        within("out", out, ref, bound)
        within("lse", lse, ref_lse, lse_bound)


def within(name, got, ref, bound):
    got = got.double().cpu()
    ok = ((got - ref).abs() <= bound) | (got == ref) | (got.isnan() & ref.isnan())
    if not bool(ok.all()):
        at = tuple(int(i) for i in (~ok).nonzero()[0])
        raise AssertionError(f"{name}: {int((~ok).sum())} of {ok.numel()} out of bounds; at {at}: {got[at]} against "
                             f"{ref[at]}, bound {bound[at]}")


class Pages:
    """The pool on lists, one sequence after the other, from the definitions."""

    def __init__(self, pages, page, seqs, max_pages):
        self.page, self.refs = page, [0] * pages
        self.table, self.held = [[0] * max_pages for _ in range(seqs)], [0] * seqs
        self.max_pages = max_pages

    def reserve(self, length, need):
        """(got, copies [(source page, target page, rows)], sequences recorded)."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        got, copies, recorded, out = [], [], [], False
        for b, (n, more) in enumerate(zip(length, need)):
            if more < 0 or not 0 <= n <= self.held[b] * self.page or n + more > self.max_pages * self.page:
                recorded.append(b)
                got.append(0)
                continue
            k, rows = divmod(n, self.page)
            copy = more > 0 and rows > 0 and self.refs[self.table[b][k]] > 1
            want = max(self.held[b], -(-(n + more) // self.page)) if more > 0 else self.held[b]
            extra = want - self.held[b] + copy
            out = out or extra > len(free)
            got.append(int(extra == 0 or not out))
            if not got[-1]:
                continue
            if copy:
                old, new = self.table[b][k], free.pop(0)
                self.table[b][k] = new
                self.refs[old] -= 1
                self.refs[new] = 1
                copies.append((old, new, rows))
            for j in range(self.held[b], want):
                self.table[b][j] = free.pop(0)
                self.refs[self.table[b][j]] = 1
            self.held[b] = want
        return got, copies, recorded

    def fork(self, src, dst, length):
        found, taken = [], set()
        for s, d in zip(src, dst):   # all are read as the call finds them
            ok = 0 <= s < len(self.held) and 0 <= d < len(self.held) and s != d and d not in taken and self.held[d] == 0 and \
                0 <= length[s] <= self.held[s] * self.page
            taken.add(d)
            if ok:
                found.append((s, d, -(-length[s] // self.page), length[s]))
        for s, d, k, n in found:
            for j in range(k):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            self.held[d], length[d] = k, n
        return len(found)

    def accept(self, ctx, path, count):
        """(after, moves [(source place, target place)] in order)."""
        after, moves = [], []
        for b, n in enumerate(count):
            p = list(range(max(n, 0))) if path is None else path[b][:max(n, 0)]
            bad = not 0 <= ctx[b] <= self.held[b] * self.page or any(y <= x for x, y in zip([-1] + p, p)) or \
                (p and ctx[b] + p[-1] >= self.held[b] * self.page)
            if bad or n < 0:
                after.append(ctx[b])
                continue
            place = lambda x: (self.table[b][x // self.page], x % self.page)
            moves += [(place(ctx[b] + x), place(ctx[b] + i)) for i, x in enumerate(p)]
            after.append(ctx[b] + n)
            while self.held[b] > -(-after[b] // self.page):
                self.held[b] -= 1
                self.refs[self.table[b][self.held[b]]] -= 1
        return after, moves

    def free(self, ids):
        for b in ids:
            if 0 <= b < len(self.held):
                for p in self.table[b][:self.held[b]]:
                    self.refs[p] -= 1
                self.held[b] = 0

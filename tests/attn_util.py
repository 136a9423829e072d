"""64-bit references and error bounds of the attention-side operators (rotary positions, cache
rows, tree attention), written from the formulas on the CPU."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def rotate_ref(x, positions, w, mag, rot, interleaved, inverse=False):
    """[tokens, heads, dim] float64: each pair turned by position * frequency, times mag."""
    y = np.array(x, np.float64)
    ang = np.asarray(positions, np.float64)[:, None] * np.asarray(w)[None, :rot // 2]
    c, s = mag * np.cos(ang)[:, None], mag * np.sin(ang)[:, None]
    if inverse:
        s = -s
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, w, mag, rot, interleaved, out_bf16, ref):
    """Error of the fp32 rotation by an fp32 table: the table entries and each of the two products
    and their sum are off by 2^-24 relative, so a channel by at most 4 * 2^-24 (|a| + |b|) mag; and
    rounding to bf16 (8 significant bits) by 2^-8 of the (erring) result."""
    x = np.abs(np.array(x, np.float64))
    both = x.copy()
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    both[..., ia] = both[..., ib] = (x[..., ia] + x[..., ib]) * mag
    e = 2.0 ** -22 * both
    return e + 2.0 ** -8 * (np.abs(ref) + e) if out_bf16 else e


def quantise_ref(x32):
    """Codes and scales of fp32 rows, as the formula has them in fp32: amax / 448, x / scale."""
    amax = x32.abs().amax(-1)
    scale = amax / np.float32(448.0)
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x32 / scale[..., None]).to(E4M3).view(torch.uint8), scale


class Pass:
    """A seeded batch for tree attention: ragged contexts and draft trees over shuffled pages."""

    def __init__(self, ctx, n, q_heads, kv_heads, dim, page, cache="bf16", q_type=torch.bfloat16, tree=True, seed=0,
                 spread=2.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.n, self.group, self.kv_heads, self.dim, self.page = list(ctx), list(n), q_heads // kv_heads, kv_heads, dim, page
        total = sum(n)
        need = [max(1, -(-(a + b) // page)) for a, b in zip(ctx, n)]
        pages = sum(need) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(ctx), max(need) + 1), 0, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.mask = None
        if tree:
            seen_all = []
            for k in n:
                seen = []
                for i in range(k):
                    parent = int(rng.integers(-1, i)) if i else -1
                    seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
                seen_all += seen
            self.mask = np.array(seen_all, np.uint64)
        self.q = (torch.randn((total, q_heads, dim), generator=g) * spread).to(q_type)
        shape = (pages, page, kv_heads, dim)
        k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        self.k_scale = self.v_scale = None
        if cache == "e4m3":
            (k, ks), (v, vs) = quantise_ref(k * (0.5 + torch.rand(shape[:3], generator=g))[..., None]), quantise_ref(
                v * torch.exp(2 * torch.randn(shape[:3], generator=g))[..., None])
            self.k_scale, self.v_scale = ks.transpose(1, 2).contiguous(), vs.transpose(1, 2).contiguous()
        else:
            t = {"bf16": torch.bfloat16, "f32": torch.float32}[cache]
            k, v = k.to(t), v.to(t)
        self.k, self.v, self.cache_type = k, v, cache

    def rows(self, name, b, h):
        """float64 [ctx + n, dim] of one sequence and cache head."""
        length = self.ctx[b] + self.n[b]
        p = np.arange(length)
        page, at = torch.from_numpy(self.table[b][p // self.page].astype(np.int64)), torch.from_numpy(p % self.page)
        x = getattr(self, name)[page, at, h]
        if self.cache_type == "e4m3":
            return x.view(E4M3).double() * getattr(self, name + "_scale")[page, h, at].double()[:, None]
        return x.double()

    def sees(self, b):
        length, n = self.ctx[b] + self.n[b], self.n[b]
        see = torch.ones((n, length), dtype=torch.bool)
        for i in range(n):
            bits = (1 << (i + 1)) - 1 if self.mask is None else int(self.mask[self.starts[b] + i])
            for j in range(n):
                see[i, self.ctx[b] + j] = bool((bits >> j) & 1)
        return see

    def reference_heads(self, heads, p_eps, out_bf16):
        """{query head: (out, lse, out bound, lse bound)} of some heads only."""
        found = {}
        for h in heads:
            one = Pass.__new__(Pass)
            one.__dict__.update(self.__dict__)
            hk = h // self.group
            one.q, one.group = self.q[:, h:h + 1], 1
            cut = lambda x, d: None if x is None else x.narrow(d, hk, 1)
            one.k, one.v = cut(self.k, 2), cut(self.v, 2)
            one.k_scale, one.v_scale = cut(self.k_scale, 1), cut(self.v_scale, 1)
            found[h] = tuple(x[:, 0] for x in one.reference(p_eps, out_bf16))
        return found

    def reference(self, p_eps, out_bf16, scale=None):
        """(out, lse, out bound, lse bound) in float64.  With s off by ds = (dim + 4) 2^-24 scale
        sum|q||k| (fp32 products summed in any order) a weight is off by 2 ds relative; exponential,
        sums and the final division add 2^-18 at most (longest sum here 2^13 terms of 2^-24 each
        would be 2^-11 at worst; errors of a pairwise or tiled sum of positive terms stay below
        2^-18); p_eps is the rounding of the weights for the product with v.  All of that scales
        sum p |v|; rounding the result to bf16 adds 2^-8 |out|."""
        total, hq = self.q.shape[:2]
        scale = self.dim ** -0.5 if scale is None else scale
        out, lse = torch.zeros((total, hq, self.dim), dtype=torch.float64), torch.full((total, hq), -np.inf, dtype=torch.float64)
        ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
        for b in range(len(self.n)):
            if self.n[b] == 0:
                continue
            see, t = self.sees(b), slice(int(self.starts[b]), int(self.starts[b + 1]))
            for h in range(hq):
                k, v = self.rows("k", b, h // self.group), self.rows("v", b, h // self.group)
                q = self.q[t, h].double()
                s = (q @ k.T * scale).masked_fill(~see, -np.inf)
                k0 = torch.where(see.any(0)[:, None], k, torch.zeros_like(k))
                ds = (self.dim + 4) * 2.0 ** -24 * scale * (q.abs() @ k0.abs().T).masked_fill(~see, 0.0).amax(-1)
                top = torch.where(see.any(-1), s.amax(-1), torch.zeros(()).double())
                e = torch.exp(s - top[:, None])
                z = e.sum(-1)
                p = e / torch.where(z > 0, z, torch.ones_like(z))[:, None]
                for i in range(p.shape[0]):   # what a token does not see is not touched
                    pi, vi = p[i][see[i]], v[see[i]]
                    out[t.start + i, h] = pi @ vi
                    ob[t.start + i, h] = (p_eps + 2 * ds[i] + 2.0 ** -18) * (pi @ vi.abs())
                lse[t, h] = torch.where(z > 0, torch.log(z) + top, torch.tensor(-np.inf).double())
                lb[t, h] = ds + 2.0 ** -20 * (1 + top.abs())
        if out_bf16:
            ob = ob + 2.0 ** -8 * (out.abs() + ob)
        return out, lse, ob, lb

    def device(self, api, dev="cuda"):
        to = lambda x: None if x is None else x.to(dev)
        cache = api.KVCache(to(self.k), to(self.v), to(self.k_scale), to(self.v_scale))
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        return dict(cache=cache, q=to(self.q), q_start=t(self.starts), ctx=t(np.array(self.ctx, np.int32)),
                    page_table=t(self.table), mask=None if self.mask is None else t(self.mask.view(np.int64)))


def weight_eps(p):
    """Rounding of the softmax weights before the product with v on the tensor cores: bf16 (2^-8)
    over a bf16 cache, fp16 (2^-11) over e4m3 codes; none on the CUDA cores.  Heads wider than 128
    and fp32 queries run there."""
    if p.q.dtype != torch.bfloat16 or p.cache_type == "f32":
        return 0.0
    return 2.0 ** -11 if p.cache_type == "e4m3" else 2.0 ** -8


def assert_within(name, got, ref, bound):
    got = got.double().cpu()
    ok = (got - ref).abs() <= bound
    ok |= (got == ref)   # infinities
    ok |= got.isnan() & ref.isnan()
    if not bool(ok.all()):
        at = tuple(int(i) for i in (~ok).nonzero()[0])
        raise AssertionError(f"{name}: {int((~ok).sum())} of {ok.numel()} out of bounds; at {at}: {got[at]} against "
                             f"{ref[at]}, bound {bound[at]}")

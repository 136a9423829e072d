"""Fork, reserve, accept and free of a pool's pages against the same steps on lists, and the rows of every
layer's cache against the moves, bit by bit."""
import random

import pytest
import torch

from latent_util import Pages
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def kv(pages, page, heads=2, dim=16, dtype="bf16", pad=0):
    """A cache with random bits; pad: rows of other strides."""
    t = {"bf16": torch.int16, "f32": torch.int32, "e4m3": torch.uint8}[dtype]
    real = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.uint8}[dtype]
    bits = lambda: torch.randint(0, 100, (pages, page + pad, heads + pad, dim), device="cuda").to(t).view(real)[:, :page, :heads]
    if dtype != "e4m3":
        return api.KVCache(bits(), bits())
    scales = lambda: torch.rand((pages, heads, page), device="cuda")
    return api.KVCache(bits(), bits(), scales(), scales())


def latent(pages, page, rank=32, rope=16, pad=0):
    return api.LatentCache(torch.randn((pages, page + pad, rank + rope), device="cuda").bfloat16()[:, :page], rank)


def parts(pool):
    """Every part of every cache as [pages, page, ...] views."""
    for c in pool.caches:
        if isinstance(c, api.LatentCache):
            yield c.rows
            continue
        yield c.k
        yield c.v
        if c.k_scale is not None:
            yield c.k_scale.transpose(1, 2)
            yield c.v_scale.transpose(1, 2)


class Both:
    """A pool on the device beside the one on lists."""

    def __init__(self, caches, seqs, max_pages):
        self.pool, c = api.page_pool(caches, seqs, max_pages), caches[0]
        self.ref = Pages(c.pages, c.page, seqs, max_pages)
        self.length = [0] * seqs

    def expect(self, pairs):
        """What the caches hold after rows moved from place to place."""
        want = [x.clone() for x in parts(self.pool)]
        before = [x.clone() for x in want]
        for (a, r), (b, s) in pairs:
            for x, y in zip(want, before):
                x[b, s] = y[a, r]
        return want

    def check(self, want, error=0):
        assert api.last_device_error(self.pool.ws) == error
        assert self.pool.refs.tolist() == self.ref.refs
        assert self.pool.held.tolist() == self.ref.held
        for b, n in enumerate(self.ref.held):
            assert self.pool.table[b, :n].tolist() == self.ref.table[b][:n]
        for x, y in zip(parts(self.pool), want):
            assert torch.equal(x.contiguous().reshape(-1).view(torch.uint8), y.contiguous().reshape(-1).view(torch.uint8))

    def reserve(self, need, error=0):
        got, copies, recorded = self.ref.reserve(self.length, need)
        want = self.expect([((a, r), (b, r)) for a, b, rows in copies for r in range(rows)])
        assert api.pages_reserve(self.pool, i32(self.length), i32(need)).tolist() == got
        self.check(want, 5 if recorded else error)
        return got, copies

    def fork(self, src, dst, error=0):
        length = i32(self.length)
        self.ref.fork(src, dst, self.length)
        want = self.expect([])
        api.pages_fork(self.pool, i32(src), i32(dst), length)
        assert length.tolist() == self.length
        self.check(want, error)

    def accept(self, path, count, error=0):
        after, moves = self.ref.accept(self.length, path, count)
        want = self.expect(moves)
        got = api.pages_accept(self.pool, i32(self.length), None if path is None else i32(path), i32(count))
        assert got.tolist() == after
        self.check(want, error)
        self.length = after

    def free(self, ids, error=0):
        length = i32(self.length)
        self.ref.free(ids)
        for b in ids:
            if 0 <= b < len(self.length):
                self.length[b] = 0
        api.pages_free(self.pool, i32(ids), length)
        assert length.tolist() == self.length
        self.check(self.expect([]), error)


@pytest.mark.parametrize("page,make", [
    (16, lambda n, p: [kv(n, p)]),
    (4, lambda n, p: [kv(n, p, 3, 16, "e4m3"), kv(n, p, 3, 16, "e4m3")]),
    (5, lambda n, p: [kv(n, p, 1, 4, "f32"), latent(n, p), kv(n, p, 2, 8, "bf16")]),
    (64, lambda n, p: [latent(n, p, 512, 64) for _ in range(3)]),
    (8, lambda n, p: [kv(n, p, 2, 16, "bf16", pad=3), latent(n, p, pad=1), kv(n, p, 2, 32, "e4m3", pad=1)]),
    (3, lambda n, p: [kv(n, p, 2, 8) for _ in range(70)]),   # more layers than one launch takes
    (8, lambda n, p: [f(n, p) for _ in range(10) for f in (kv, latent, lambda n, p: kv(n, p, 1, 64, "e4m3"))]),   # shapes in turn
])
def test_a_run_of_all_steps(page, make):
    """Rounds of drafting, acceptance, branching and giving up, with random paths."""
    rng = random.Random(page)
    seqs, max_pages = 9, -(-200 // page) + 1
    b = Both(make(40 + 900 // page, page), seqs, max_pages)
    assert b.reserve([rng.randint(1, 60) if i < 4 else 0 for i in range(seqs)])[0] == [1] * seqs
    b.accept(None, [min(rng.randint(0, 40), h * page, 64) for h in b.ref.held])
    for _ in range(6):
        empty = [i for i in range(seqs) if b.ref.held[i] == 0]
        owners = [i for i in range(seqs) if b.ref.held[i] > 0]
        rng.shuffle(empty)
        k = min(len(empty), 3)
        if owners and k:
            b.fork([rng.choice(owners) for _ in range(k)], empty[:k])
        need = [rng.randint(0, 30) for _ in range(seqs)]
        b.reserve(need)
        path, count = [], []
        for i in range(seqs):
            room = min(30, b.ref.held[i] * page - b.length[i], 200 - b.length[i])
            n = rng.randint(0, min(8, max(0, room))) if need[i] > 0 else 0
            p = sorted(rng.sample(range(room), n))
            path.append(p + [rng.randint(-5, 99) for _ in range(8 - n)])   # what lies behind the count is not read
            count.append(n if rng.random() < 0.9 else -1)
        b.accept(path, count)
        b.free(rng.sample(range(seqs), 2) + [-1])


def test_shared_page_goes_to_the_last_holder():
    b = Both([kv(30, 8), latent(30, 8)], 6, 5)
    b.reserve([11, 0, 0, 0, 0, 0])
    b.accept(None, [11, 0, 0, 0, 0, 0])
    b.fork([0, 0, 0], [1, 2, 3])
    assert b.ref.refs[0] == b.ref.refs[1] == 4
    # three of four write: all take a copy; then the last holder has it alone
    got, copies = b.reserve([0, 1, 1, 1, 0, 0])
    assert len(copies) == 3
    assert b.reserve([1, 0, 0, 0, 0, 0])[1] == []
    b.free([1, 2, 3])
    b.fork([0, 0], [4, 5])
    got, copies = b.reserve([3, 0, 0, 0, 3, 3])   # all three: the last of them keeps the page
    assert len(copies) == 2 and got == [1] * 6


def test_pages_run_out():
    b = Both([kv(10, 4)], 5, 9)
    # 3 + 3 pages fit, the third sequence's 6 do not, nor do the last one's 2 behind it; nothing needed is met
    assert b.reserve([12, 9, 24, 0, 5])[0] == [1, 1, 0, 1, 0]
    b.free([0])
    assert b.reserve([0, 0, 24, 0, 0])[0] == [1, 1, 1, 1, 1]
    assert b.reserve([0, 0, 0, 0, 8])[0] == [1, 1, 1, 1, 0]
    # a shared page cannot be copied, and the next sharer must not take it for its own
    b = Both([kv(2, 4)], 3, 4)
    b.reserve([6, 0, 0])
    b.accept(None, [6, 0, 0])
    b.fork([0, 0], [1, 2])
    assert b.reserve([1, 1, 1])[0] == [0, 0, 0]
    b.free([0])
    b.free([1])
    assert b.reserve([0, 0, 1])[0] == [1, 1, 1]


def test_many_sequences_and_pages():
    """All threads of the bookkeeping, and free pages beyond its first step."""
    pages = 70001
    b = Both([latent(pages, 8, 8, 8)], 1024, 80)
    rng = random.Random(1)
    b.reserve([rng.randint(0, 590) for _ in range(1024)])
    assert sum(b.ref.held) > 32768
    b.length = [h * 8 - rng.randint(0, 7) if h else 0 for h in b.ref.held]
    b.free(rng.sample(range(1024), 300))
    free = [i for i in range(1024) if b.ref.held[i] == 0]
    owners = [i for i in range(1024) if b.ref.held[i] > 0]
    b.fork([rng.choice(owners) for _ in free], free)
    b.reserve([rng.randint(0, 40) if b.length[i] < 600 else 0 for i in range(1024)])


def test_bad_indices_are_recorded_and_leave_their_sequence():
    b = Both([kv(20, 4), latent(20, 4)], 4, 6)
    b.reserve([9, 5, 0, 0])
    b.accept(None, [9, 5, 0, 0])
    b.reserve([-1, 3, 0, 0])
    b.reserve([2, 100, 0, 0])                      # beyond the table
    b.fork([0, 1, 0, 7, 0], [2, 2, 0, 3, -1], 5)     # the same target twice, itself, no such sequence
    assert b.ref.held[2] == 3 and b.ref.held[3] == 0
    b.free([3, 9], 5)
    b.reserve([4, 4, 4, 0])
    b.accept([[1, 1], [2, 1], [0, 2], [0, 0]], [2, 2, 2, 0], 5)      # paths that do not ascend
    b.accept([[0, 3], [-1, 2], [0, 90], [0, 0]], [2, 2, 2, -3], 5)   # outside the pages held
    b.accept([[0, 2], [1, 2], [0, 1], [0, 1]], [3, 0, 2, 1], 5)      # longer than a path, nothing held
    b.free([0, 0, 1, 0])                            # one sequence named three times
    assert sum(b.ref.refs) == b.ref.held[2]
    b.free([2])
    assert sum(b.ref.refs) == 0


def test_rows_do_not_move_into_shared_pages():
    b = Both([kv(20, 4), latent(20, 4)], 3, 6)
    b.reserve([12, 0, 0])
    b.accept(None, [6, 0, 0])
    b.fork([0], [1])
    # sequence 0 drafts without reserving: its part-filled page is the other's too
    before = b.expect([])
    after = api.pages_accept(b.pool, i32(b.length), i32([[1], [0], [0]]), i32([1, -1, -1]))
    assert after.tolist() == b.length
    b.check(before, 5)
    b.reserve([4, 0, 0])
    b.accept([[1], [0], [0]], [1, -1, -1])


def test_many_forks_at_once():
    """More pairs than a CTA copies, equal targets among them, on one workspace."""
    pages = 600
    b = Both([latent(pages, 4, 8, 8)], 400, 8)
    rng = random.Random(2)
    b.reserve([rng.randint(0, 24) if i < 100 else 0 for i in range(400)])
    b.length = [h * 4 - rng.randint(0, 3) if h else 0 for h in b.ref.held]
    for _ in range(3):
        free = [i for i in range(400) if b.ref.held[i] == 0]
        dst = rng.sample(free, 150) + rng.sample(range(400), 50)
        src = [rng.randrange(100) for _ in dst]
        b.fork(src, dst, 5)
        b.free([d for d in dst if d >= 100])


def test_lengths_in_place_and_graphs():
    caches = [kv(40, 8) for _ in range(2)]
    pool = api.page_pool(caches, 3, 10)
    length, need, got = i32([0, 0, 0]), i32([6, 6, 6]), i32([0, 0, 0])
    path, count = i32([[0, 2, 5], [0, 1, 2], [1, 3, 4]]), i32([3, 2, 3])
    api.pages_reserve(pool, length, need, got)      # loads the kernels
    api.pages_accept(pool, length, path, count, after=length)
    assert length.tolist() == [3, 2, 3]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.pages_reserve(pool, length, need, got)
        api.pages_accept(pool, length, path, count, after=length)
    ref = Pages(40, 8, 3, 10)
    steps = [0, 0, 0]
    for k in range(6):
        if k:
            graph.replay()
        ref.reserve(steps, [6, 6, 6])
        steps = ref.accept(steps, path.tolist(), count.tolist())[0]
        assert length.tolist() == steps and pool.held.tolist() == ref.held and pool.refs.tolist() == ref.refs
    assert api.last_device_error(pool.ws) == 0

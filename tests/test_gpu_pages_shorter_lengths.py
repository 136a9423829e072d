"""Reserve for sequences whose length was lowered after a fork: pages behind it that others hold are replaced before
they are written."""
import random

import pytest
import torch

from latent_util import Pages
from moe_speculative_decoding_gb300 import api
from test_gpu_pages import Both, i32, kv, latent

pytestmark = pytest.mark.gpu


class Lists(Pages):
    def reserve(self, length, need):
        """(got, copies [(source page, target page, rows)], sequences recorded): one sequence after the other.  Of the
        pages to be written that others held before the call, the one with position `length` inside is copied
        as long as others than those that have copied it hold it, and those behind are replaced."""
        found = list(self.refs)
        free = [p for p, r in enumerate(found) if r == 0]
        given, after = {}, list(found)   # copies taken of a page; holders after the call
        got, copies, recorded, out = [], [], [], False
        for b, (n, more) in enumerate(zip(length, need)):
            if more < 0 or not 0 <= n <= self.held[b] * self.page or n + more > self.max_pages * self.page:
                recorded.append(b)
                got.append(0)
                continue
            if more == 0:
                got.append(1)
                continue
            first, rows = divmod(n, self.page)
            pages = -(-(n + more) // self.page)
            behind = [j for j in range(first + (rows > 0), min(self.held[b], pages)) if found[self.table[b][j]] > 1]
            old = self.table[b][first] if rows else None
            copy = rows > 0 and found[old] > 1 and found[old] - given.get(old, 0) > 1
            extra = int(copy) + len(behind) + max(0, pages - self.held[b])
            out = out or extra > len(free)
            got.append(int(extra == 0 or not out))
            if not got[-1]:
                continue
            if copy:
                given[old] = given.get(old, 0) + 1
                copies.append((old, free[0], rows))
                behind = [first] + behind
            for j in behind:
                after[self.table[b][j]] -= 1
                self.table[b][j] = free.pop(0)
                after[self.table[b][j]] = 1
            for j in range(self.held[b], pages):
                self.table[b][j] = free.pop(0)
                after[self.table[b][j]] = 1
            self.held[b] = max(self.held[b], pages)
        self.refs = after
        return got, copies, recorded


class Run(Both):
    def __init__(self, caches, seqs, max_pages):
        super().__init__(caches, seqs, max_pages)
        c = caches[0]
        self.ref = Lists(c.pages, c.page, seqs, max_pages)

    def reserve(self, need, error=0):
        got, copies = super().reserve(need, error)
        for b, (n, more) in enumerate(zip(self.length, need)):   # what may be written now is nobody else's
            if got[b] and more:
                for j in range(n // self.ref.page, -(-(n + more) // self.ref.page)):
                    assert int(self.pool.refs[int(self.pool.table[b, j])]) == 1
        return got, copies


def test_lowered_to_a_boundary_and_inside_a_page():
    for length in (8, 5):
        b = Run([kv(30, 4), latent(30, 4)], 3, 6)
        b.reserve([10, 0, 0])
        b.length = [10, 0, 0]
        b.fork([0, 0], [1, 2])
        b.length[0] = length
        got, copies = b.reserve([6, 0, 0])     # pages 2 (and 1) were all three's
        assert got == [1, 1, 1] and len(copies) == (length % 4 > 0)
        assert b.ref.refs[2] == 2
        b.length[2] = 0
        b.reserve([0, 2, 10])                   # one copies a page's rows, one begins anew and keeps none
    assert api.last_device_error(b.pool.ws) == 0


def test_all_give_up_a_page_at_once():
    """Two that share a page behind their lengths: neither keeps it, and it is free after the call."""
    b = Run([kv(30, 4)], 2, 6)
    b.reserve([12, 0])
    b.length = [12, 0]
    b.fork([0], [1])
    b.length = [8, 8]
    b.reserve([1, 1])
    assert b.ref.refs[2] == 0
    # one copies the first rows of a page that another replaces
    b = Run([kv(30, 4)], 2, 6)
    b.reserve([12, 0])
    b.length = [12, 0]
    b.fork([0], [1])
    b.length = [10, 8]
    assert len(b.reserve([1, 1])[1]) == 1
    assert b.ref.refs[2] == 0


def test_spare_pages_are_left_until_they_are_written():
    b = Run([kv(30, 4)], 2, 6)
    b.reserve([20, 0])
    b.length = [20, 0]
    b.fork([0], [1])
    b.length[0] = 4
    b.reserve([3, 0])
    assert b.ref.refs[1:5] == [1, 2, 2, 2]
    b.reserve([5, 0])
    assert b.ref.refs[1:5] == [1, 1, 2, 2]


def test_pages_run_out():
    b = Run([kv(7, 4)], 3, 6)
    b.reserve([16, 0, 0])
    b.length = [16, 0, 0]
    b.fork([0, 0], [1, 2])
    b.length = [4, 2, 16]
    # 3 free: the first takes two, the second would take two, the third one needs one
    assert b.reserve([8, 6, 1])[0] == [1, 0, 0]
    assert b.reserve([0, 0, 1])[0] == [1, 1, 1]


@pytest.mark.parametrize("page,seed", [(1, 1), (4, 2), (4, 3), (16, 4), (5, 5)])
def test_random_rounds(page, seed):
    rng = random.Random(seed)
    seqs, most = 12, 60 // page + 4
    b = Run([kv(seqs * most // 2, page, 1, 16), latent(seqs * most // 2, page, 8, 8)], seqs, most)
    b.reserve([rng.randint(1, 60) if i < 3 else 0 for i in range(seqs)])
    b.length = [h * page for h in b.ref.held]
    for _ in range(12):
        empty = [i for i in range(seqs) if b.ref.held[i] == 0]
        owners = [i for i in range(seqs) if b.ref.held[i] > 0]
        rng.shuffle(empty)
        if owners and empty:
            b.fork([rng.choice(owners) for _ in empty[:6]], empty[:6])
        for i in range(seqs):
            if rng.random() < 0.5:
                b.length[i] = rng.randint(0, b.length[i])
        b.reserve([rng.randint(0, max(0, min(30, most * page - b.length[i]))) if rng.random() < 0.7 else 0 for i in range(seqs)])
        b.length = [rng.randint(n, b.ref.held[i] * page) for i, n in enumerate(b.length)]
        b.free(rng.sample(range(seqs), 3))
    assert sum(r > 0 for r in b.ref.refs) == len({p for i in range(seqs) for p in b.ref.table[i][:b.ref.held[i]]})

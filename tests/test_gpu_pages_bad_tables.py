"""Page numbers and counts of held pages that are out of range: the sequence that has them is recorded and left as it
was by every call, and the others are served."""
import pytest
import torch

from moe_speculative_decoding_gb300 import api
from test_gpu_pages import Both, i32, kv, latent, parts

pytestmark = pytest.mark.gpu
BAD_ID = 5
NUMBERS = [-1, 20, 2 ** 31 - 1, -2 ** 31]


class State:
    """Everything that a call on a pool may change."""

    def __init__(self, pool, *more):
        self.all = [pool.refs, pool.held, pool.table, *more, *parts(pool)]
        self.before = [x.clone() for x in self.all]

    def unchanged(self):
        return all(torch.equal(x.contiguous().view(-1).view(torch.uint8), y.contiguous().view(-1).view(torch.uint8))
                   for x, y in zip(self.all, self.before))


def pool_of(seqs, reserve, lengths):
    b = Both([kv(20, 4), latent(20, 4), kv(20, 4, 2, 16, "e4m3")], seqs, 6)
    b.reserve(reserve)
    b.length = lengths
    return b


@pytest.mark.parametrize("number", NUMBERS)
def test_reserve(number):
    b = pool_of(2, [16, 0], [6, 0])
    b.pool.table[0, 1] = number
    state = State(b.pool)
    assert api.pages_reserve(b.pool, i32([6, 0]), i32([4, 0])).tolist() == [0, 1]
    assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()


@pytest.mark.parametrize("number", NUMBERS)
@pytest.mark.parametrize("where", [1, 2, 3])   # where rows move to; given up alone; where rows come from, and given up
def test_accept(number, where):
    # sequence 0: positions 7 and 13 (pages 1 and 3) move to 6 and 7 (page 1); pages 2 and 3 are given up
    b = pool_of(2, [16, 16], [6, 6])
    good = int(b.pool.table[0, where])
    b.pool.table[0, where] = number
    state = State(b.pool)
    after = api.pages_accept(b.pool, i32([6, 6]), i32([[1, 7], [0, 0]]), i32([2, -1]))
    assert api.last_device_error(b.pool.ws) == BAD_ID
    assert after.tolist() == [6, 6] and state.unchanged()
    # the other sequence is served
    b.pool.table[0, where] = good
    after, moves = b.ref.accept([6, 6], [[0, 0], [1, 7]], [-1, 2])
    want = b.expect(moves)
    b.pool.table[0, where] = number
    got = api.pages_accept(b.pool, i32([6, 6]), i32([[1, 7], [1, 7]]), i32([2, 2]))
    assert got.tolist() == after
    b.pool.table[0, where] = good
    b.check(want, BAD_ID)


@pytest.mark.parametrize("number", NUMBERS)
def test_accept_that_moves_nothing(number):
    b = pool_of(2, [16, 16], [6, 6])
    b.pool.table[0, 3] = number
    state = State(b.pool)
    for path in (None, i32([[0, 1], [0, 1]])):
        after = api.pages_accept(b.pool, i32([6, 6]), path, i32([2, -1]))
        assert api.last_device_error(b.pool.ws) == BAD_ID
        assert after.tolist() == [6, 6] and state.unchanged()


@pytest.mark.parametrize("number", NUMBERS)
@pytest.mark.parametrize("pairs", [1, 60])   # one CTA, several
def test_fork(number, pairs):
    seqs = 2 + 2 * pairs
    b = pool_of(seqs, [16, 16] + [0] * 2 * pairs, [14, 9] + [0] * 2 * pairs)
    good = int(b.pool.table[0, 2])
    src, dst = [0] * pairs + [1] * pairs, list(range(2, seqs))
    length = i32(b.length)
    b.pool.table[0, 2] = number
    state = State(b.pool, length)
    api.pages_fork(b.pool, i32(src[:pairs]), i32(dst[:pairs]), length)
    assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()
    # those of the other sequence are served beside them
    refused = b.pool.table[2:2 + pairs].clone()
    b.ref.fork(src[pairs:], dst[pairs:], b.length)
    api.pages_fork(b.pool, i32(src), i32(dst), length)
    assert length.tolist() == b.length and torch.equal(b.pool.table[2:2 + pairs], refused)
    b.pool.table[0, 2] = good
    b.check(b.expect([]), BAD_ID)
    # a shorter source, whose bad number lies behind it
    length[0] = b.length[0] = 8
    b.pool.table[0, 2] = number
    b.ref.fork([0], [2], b.length)
    api.pages_fork(b.pool, i32([0]), i32([2]), length)
    b.pool.table[0, 2] = good
    assert length.tolist() == b.length
    b.check(b.expect([]))


@pytest.mark.parametrize("number", NUMBERS)
def test_free(number):
    b = pool_of(3, [16, 16, 3], [14, 9, 3])
    good = int(b.pool.table[0, 1])
    b.pool.table[0, 1] = number
    length = i32(b.length)
    state = State(b.pool, length)
    for ids in ([0], [0, 0, 0]):
        api.pages_free(b.pool, i32(ids), length)
        assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()
    b.ref.free([1, 2])
    api.pages_free(b.pool, i32([0, 1, 0, 2, 1]), length)
    assert length.tolist() == [14, 0, 0]
    b.pool.table[0, 1] = good
    b.check(b.expect([]), BAD_ID)


@pytest.mark.parametrize("held", [-1, 7, 2 ** 31 - 1, -2 ** 31])
def test_held_out_of_range(held):
    b = pool_of(3, [16, 16, 0], [14, 9, 0])
    b.pool.held[0] = held
    length = i32(b.length)
    state = State(b.pool, length)
    api.pages_free(b.pool, i32([0, 0]), length)
    assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()
    api.pages_fork(b.pool, i32([0]), i32([2]), length)
    assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()
    assert api.pages_accept(b.pool, length, i32([[1], [0], [0]]), i32([1, -1, -1])).tolist() == b.length
    assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()
    assert api.pages_reserve(b.pool, length, i32([4, 0, 0])).tolist() == [0, 1, 1]
    assert api.last_device_error(b.pool.ws) == BAD_ID and state.unchanged()

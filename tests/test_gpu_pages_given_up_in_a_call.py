"""Acceptance where one sequence gives up a page that another would move rows into in the same call: holders count as
the call finds them, whichever comes first."""
import pytest
import torch

from moe_speculative_decoding_gb300 import api
from test_gpu_pages import i32, kv, latent, parts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [40, 12000])   # together on the device, and one after the other
@pytest.mark.parametrize("first", ["gives", "takes"])
def test_holders_are_those_before_the_call(first, pairs):
    """Pairs of which one sequence moves a row out of a page that it shares and gives that up, and the other would move
    a row within it."""
    page, k = 4, torch.arange(pairs, dtype=torch.int32, device="cuda")
    seqs = torch.arange(2 * pairs, device="cuda")
    gives, takes = (seqs[:pairs], seqs[pairs:]) if first == "gives" else (seqs[pairs:], seqs[:pairs])
    pool = api.page_pool([kv(4 * pairs, page, 2, 64), latent(4 * pairs, page)], 2 * pairs, 3)
    # both hold page 4 k + 1 as their last one: the one's pages are 4 k, 4 k + 1, the other's 4 k + 2, 4 k + 1
    pool.table[gives, 0], pool.table[takes, 0] = 4 * k, 4 * k + 2
    pool.table[gives, 1] = pool.table[takes, 1] = 4 * k + 1
    pool.refs.copy_(i32([1, 2, 1, 0]).repeat(pairs))
    pool.held.fill_(2)
    # the giver keeps its position 1 and its position 4 (of the shared page) behind it; the taker, of position 5, makes 4
    def both(give, take):
        x = torch.empty((2 * pairs, *i32(give).shape), dtype=torch.int32, device="cuda")
        x[gives], x[takes] = i32(give), i32(take)
        return x
    ctx, path = both(1, 4), both([0, 3], [1, 0])
    want = [x.clone() for x in parts(pool)]
    for x in want:
        x[4 * k.long(), 2] = x[4 * k.long() + 1, 0]
    after = api.pages_accept(pool, ctx, path, both(2, 1))
    assert api.last_device_error(pool.ws) == 5
    assert torch.equal(after, both(3, 4)) and torch.equal(pool.held, both(1, 2))
    assert torch.equal(pool.refs, i32([1, 1, 1, 0]).repeat(pairs))
    for x, y in zip(parts(pool), want):
        assert torch.equal(x.contiguous().view(-1).view(torch.uint8), y.contiguous().view(-1).view(torch.uint8))
    # now the page is the other's alone
    after = api.pages_accept(pool, ctx, path, both(-1, 1))
    assert api.last_device_error(pool.ws) == 0 and torch.equal(after, both(1, 5))


@pytest.mark.parametrize("caches", [1, 0, 12])   # launches of the rows' kernel: one, none, one for each of twelve shapes
def test_pages_are_given_up_once(caches):
    """The counts go down once, however many caches there are (none: by the C interface alone)."""
    pool = api.page_pool([kv(40, 4, 1 + i % 2, 16 * (1 + i // 2)) for i in range(max(1, caches))], 3, 6)
    api.pages_reserve(pool, i32([0] * 3), i32([20, 12, 16]))
    if caches == 0:
        empty = api.CachesDesc(None, None, 0, 0)
        pool._caches, pool.caches_address = empty, api.ctypes.addressof(empty)
    after = api.pages_accept(pool, i32([2, 3, 1]), i32([[0, 5], [0, 1], [2, 3]]), i32([2, 2, 1]))
    assert after.tolist() == [4, 5, 2] and pool.held.tolist() == [1, 2, 1]
    assert pool.refs[:12].tolist() == [1, 0, 0, 0, 0, 1, 1, 0, 1, 0, 0, 0]
    assert api.last_device_error(pool.ws) == 0

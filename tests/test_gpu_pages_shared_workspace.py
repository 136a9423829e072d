"""Forks on a workspace that other calls have used before."""
import pytest
import torch

from latent_util import LatentPass
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_forks_after_attention_on_one_workspace():
    """100 pairs take several CTAs, whose last one must not go by what an attention call left behind the header."""
    p = LatentPass([5000], [4], 16, 512, 64, 64, seed=1)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 4, 1, 16)
    pool = api.page_pool([d["cache"]], 101, 4)
    assert ws.numel() >= pool.ws_bytes
    pool.ws, pool.ws_bytes = ws, ws.numel()
    length = i32([100] + [0] * 100)
    assert api.pages_reserve(pool, i32([0] * 101), length).tolist() == [1] * 101
    for _ in range(3):
        out, lse = api.latent_attention(**d, return_lse=True, max_tokens=4, ws=ws)
        api.pages_fork(pool, i32([0] * 100), i32(list(range(1, 101))), length)
        assert api.last_device_error(ws) == 0
        assert pool.held.tolist() == [2] * 101 and length.tolist() == [100] * 101
        assert pool.refs[:2].tolist() == [101, 101] and pool.table[:, :2].tolist() == [[0, 1]] * 101
        api.pages_free(pool, i32(list(range(1, 101))), length)
    p.check(api, out, lse)


def test_captured_forks_of_several_ctas():
    """Attention, 100 forks and their end in one graph, on one workspace, replayed."""
    p = LatentPass([5000], [4], 16, 512, 64, 64, seed=2)
    d = p.device(api)
    ws = api.latent_attention_workspace(d["cache"], 4, 1, 16)
    pool = api.page_pool([d["cache"]], 101, 4)
    pool.ws, pool.ws_bytes = ws, ws.numel()
    length = i32([100] + [0] * 100)
    api.pages_reserve(pool, i32([0] * 101), length)
    src, dst, seen = i32([0] * 100), i32(list(range(1, 101))), torch.zeros((101, 3), dtype=torch.int32, device="cuda")
    out, lse = torch.zeros((4, 16, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 16), device="cuda")

    def steps():
        api.latent_attention(**d, out=out, lse=lse, max_tokens=4, ws=ws)
        api.pages_fork(pool, src, dst, length)
        seen[:, 0].copy_(pool.held)
        seen[:, 1].copy_(length)
        api.pages_free(pool, dst, length)
        seen[:, 2].copy_(pool.held)

    steps()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
        steps()
    for _ in range(3):
        seen.zero_()
        out.zero_()
        graph.replay()
        assert seen.tolist() == [[2, 100, 2]] + [[2, 100, 0]] * 100
        assert pool.refs[:2].tolist() == [1, 1] and length.tolist() == [100] + [0] * 100
        p.check(api, out, lse)
    assert api.last_device_error(ws) == 0


def test_two_pools_at_once():
    """Two pools, each with its workspace and stream, side by side."""
    def steps(pool, length, more, src, dst, rounds):
        for _ in range(rounds):
            api.pages_reserve(pool, length, more)
            api.pages_accept(pool, length, path, count, after=length)
            api.pages_fork(pool, src, dst, length)
            api.pages_reserve(pool, length, more)
            api.pages_free(pool, dst, length)

    n = 100
    path, count = i32([[0, 2]] * 2 * n), i32([2] * n + [-1] * n)
    more, src, dst = i32([3] * n + [0] * n), i32(list(range(n))), i32(list(range(n, 2 * n)))
    make = lambda k: (api.page_pool([api.LatentCache(torch.arange(4000 * 4 * 16, device="cuda").view(4000, 4, 16).bfloat16() * (k + 1), 8)], 2 * n, 20),
                      i32([0] * 2 * n))
    alone = [make(0), make(1)]
    for x in alone:
        steps(*x, more, src, dst, 12)
    torch.cuda.synchronize()
    both, streams = [make(0), make(1)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(12):
        for x, s in zip(both, streams):
            with torch.cuda.stream(s):
                steps(*x, more, src, dst, 1)
    torch.cuda.synchronize()
    for (a, la), (b, lb) in zip(alone, both):
        assert torch.equal(la, lb) and torch.equal(a.refs, b.refs) and torch.equal(a.held, b.held) and torch.equal(a.table, b.table)
        assert torch.equal(a.caches[0].rows, b.caches[0].rows)
        assert api.last_device_error(a.ws) == 0 and api.last_device_error(b.ws) == 0
        assert la.tolist() == [24] * n + [0] * n

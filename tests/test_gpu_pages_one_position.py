"""Pages of one position: a row's scales of all heads then lie together, at any address that is a multiple of 4."""
import random

import pytest
import torch

from moe_speculative_decoding_gb300 import api
from test_gpu_pages import Both, kv, latent

pytestmark = pytest.mark.gpu


def codes(pages, heads, dim, offset):
    """An e4m3 cache with pages of one position, its scales `offset` floats behind a 16-byte boundary."""
    bits = lambda: torch.randint(0, 100, (pages, 1, heads, dim), device="cuda").to(torch.uint8)
    scales = lambda: torch.rand(pages * heads + offset, device="cuda")[offset:].view(pages, heads, 1)
    return api.KVCache(bits(), bits(), scales(), scales())


@pytest.mark.parametrize("make", [
    lambda n: [codes(n, 4, 16, 1)], lambda n: [codes(n, 8, 32, 3), codes(n, 8, 32, 2)], lambda n: [codes(n, 4, 16, 0)],
    lambda n: [codes(n, 3, 16, 1)], lambda n: [codes(n, 1, 16, 1)], lambda n: [kv(n, 1, 4, 16), latent(n, 1), codes(n, 12, 16, 1)]])
def test_pages_of_one_position(make):
    rng = random.Random(1)
    b = Both(make(300), 5, 50)
    b.reserve([9, 20, 1, 0, 0])
    b.accept(None, [9, 17, 1, -1, -1])
    b.fork([0, 1], [3, 4])
    for _ in range(3):
        b.reserve([8] * 5)
        b.accept([sorted(rng.sample(range(8), 4)) for _ in range(5)], [4, 3, 0, 4, 1])
    b.free([1, 3])

"""The example of a whole verification pass: speculative rounds over trees must leave the cache as a
prefill of the accepted tokens does."""
import importlib.util
import os

import pytest
import torch

from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "verify_pass.py")
    spec = importlib.util.spec_from_file_location("verify_pass", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rounds_agree_with_a_prefill_of_their_tokens(example, cache):
    """Drafts put the greedy tokens of a first run on different branches, so that paths of several
    nodes are accepted and moved.  Afterwards the logits that follow the last seen token are compared
    with a fresh prefill's: the same model in other passes, up to roundings that may swap an expert
    (16 bits in and between the layers), so by direction: cosine above 0.98, where
    the other sequences' logits are clearly elsewhere."""
    prompts = torch.randint(example.VOCAB, (3, 70), generator=torch.Generator().manual_seed(2)).cuda()
    plain, _ = example.decode(example.Model(3, cache=cache), prompts, 8, seed=3)

    def guess(trees, tokens):
        for b, t in enumerate(tokens):
            rest = plain[b][len(t) - 70:]
            for node, k in ((1, 0), (3, 1), (6, 2)):   # the root's child, its second child, that one's first
                if k < len(rest):
                    trees[b, node] = rest[k]

    model = example.Model(3, cache=cache)
    example.model_guess = guess
    try:
        out, logits = example.decode(model, prompts, 3, seed=4)
    finally:
        example.model_guess = None
    assert api.last_device_error(model.attn_ws) == 0 and api.last_device_error(model.ws) == 0
    assert max(len(o) for o in out) > 4   # paths longer than a node
    for b in range(3):
        seen = torch.cat([prompts[b], torch.tensor(out[b][:-1], device="cuda")])[None]
        fresh = example.Model(1, cache=cache)
        ref = example.prefill(fresh, seen)[0]
        near = torch.nn.functional.cosine_similarity(logits, ref[None], dim=1)
        assert near[b].item() > 0.98
        assert max(near[i].item() for i in range(3) if i != b) < 0.9   # the other sequences'


def test_rotation_gradient(example):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(9, 4, 64, device="cuda", generator=g, requires_grad=True)
    up = torch.randn(9, 4, 64, device="cuda", generator=g)
    positions = torch.randint(500, (9,), device="cuda", generator=g).int()
    table = api.rope_table(500, *api.rope_frequencies(64))
    (example.Rotary.apply(x, positions, table) * up).sum().backward()
    want = api.rope(up, None, positions, table, inverse=True)[0]
    assert torch.equal(x.grad, want)
    # the scalar product of the gradient with a step is the difference it makes (fp32, 2304 terms)
    step = torch.randn(9, 4, 64, device="cuda", generator=g)
    f = lambda y: (api.rope(y, None, positions, table)[0].double() * up.double()).sum()
    with torch.no_grad():
        diff = f(x + step) - f(x)
    assert abs((x.grad.double() * step.double()).sum() - diff) < 1e-3

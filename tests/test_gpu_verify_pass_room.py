"""The example refuses to go past its cache on the host, before anything indexes its page table."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "verify_pass.py")
    spec = importlib.util.spec_from_file_location("verify_pass", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.PAGES_EACH = 2   # 128 places a sequence
    return mod


def test_rounds_and_prompts_that_do_not_fit(example):
    prompts = torch.randint(example.VOCAB, (2, 122), generator=torch.Generator().manual_seed(2)).cuda()
    model = example.Model(2)
    with pytest.raises(ValueError, match="130 places"):
        example.decode(model, prompts, 1)
    with pytest.raises(ValueError, match="129 places"):
        example.prefill(model, prompts.repeat(1, 2)[:, :129])
    out, _ = example.decode(model, prompts[:, :112], 2)   # 112 + 8, and at most 8 more
    assert all(len(o) >= 3 for o in out)
    torch.cuda.synchronize()

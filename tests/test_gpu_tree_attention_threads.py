"""Calls of several host threads, each on its own stream."""
import threading

import pytest
import torch

from attn_util import Pass, assert_within
from moe_speculative_decoding_gb300 import api

pytestmark = pytest.mark.gpu


def test_wide_heads_from_two_threads():
    """Heads of 256 and of 192 channels need different amounts of shared memory of one kernel: neither
    call may take away what the other has asked for."""
    passes = [Pass([20], [2], 2, 1, dim, 8, "f32", q_type=torch.float32, seed=dim) for dim in (256, 192)]
    outs, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                args = passes[i].device(api)
                ws = api.tree_attention_workspace(args["cache"], 2, 1, 2)
                for _ in range(3000):
                    outs[i] = api.tree_attention(**args, ws=ws)
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for p, out in zip(passes, outs):
        ref, _, bound, _ = p.reference(0.0, False)
        assert_within("out", out, ref, bound)

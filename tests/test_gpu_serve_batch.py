"""The adapters, the attention with sinks and the verification together, as a serving step uses them: the example's batch
against the same steps in plain torch, and every token against the 64-bit oracle."""
import os
import sys

import numpy as np
import pytest

from oracle import requests as o

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kw", [dict(), dict(requests=1, drafts=0, steps=3, prompt=1), dict(requests=9, drafts=5, steps=2),
                                dict(requests=3, dim=128, q_heads=4, kv_heads=4, window=20, sinks=40, rank=70, vocab=1500)])
def test_the_example_batch(kw):
    import serve_batch
    worst, taken, offered, calls = serve_batch.run(seed=5, **kw)
    # values of order 1 to 4 in fp16 (2^-11 each; qkv is rounded before and after the adapters), sums of hidden terms in fp32
    assert worst[0] < 8e-3 and worst[1] < 4e-3 and worst[2] < 1.2e-2
    assert 0 <= taken <= offered
    for probs, draft, ids, offsets, accept, pick, out, accepted in calls:
        host = [None if t is None else t.cpu().numpy() for t in (probs, draft, ids, accept, pick)]
        want, counts = o.verify(host[0], host[1], host[2], offsets, host[3], host[4], np.full(len(host[2]), 77, np.int32))
        assert out.cpu().numpy().tolist() == want.tolist() and accepted.cpu().numpy().tolist() == counts.tolist()

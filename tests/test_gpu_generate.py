"""The generation example on the GPU (gpu): the cache carries a sequence as a
whole prompt pass does, and eviction keeps lengths within their limit."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_steps_give_the_logits_of_a_whole_pass():
    import generate as g
    model = g.Decoder()
    rng = np.random.default_rng(3)
    seqs = [rng.integers(0, g.VOCAB, n) for n in (9, 67)]
    whole = g.Cache(8, 2, 80)
    want = g.forward(model, whole, g._int32(np.concatenate(seqs)), [len(s) for s in seqs])
    parts = g.Cache(8, 2, 80)
    g.forward(model, parts, g._int32(np.concatenate([s[:-3] for s in seqs])), [len(s) - 3 for s in seqs])
    for i in (3, 2, 1):
        got = g.forward(model, parts, g._int32([s[-i] for s in seqs]), [1, 1])
    torch.cuda.synchronize()
    # the same cache values and products; attention's sums are taken in another order, then rounded to
    # bf16 (2^-8 of a value now and then one step off) through two layers: a few per cent of the logits' spread at most
    err = (got - want).float().norm() / want.float().norm()
    assert float(err) < 0.03, float(err)
    assert whole.lens == parts.lens == [9, 67]


def test_generation_with_eviction():
    import generate as g
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, g.VOCAB, n).tolist() for n in (5, 70, 119)]
    texts, cache = g.generate(prompts, 25, keep=96, limit=128)
    again, _ = g.generate(prompts, 25, keep=96, limit=128)
    assert texts == again
    assert all(0 <= t < g.VOCAB for row in texts for t in row)
    assert max(cache.lens) <= 128 and cache.lens[0] == 5 + 25 - 1

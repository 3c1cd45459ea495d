"""A run of the verify round's calls together on the GPU (gpu), by the example that
makes one: a captured round repeats the eager one bit for bit, the kept tokens
are those that the decoder chooses by itself, and pages come back."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import draft as odraft

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

PENALTIES = dict(repetition=1.1, presence=0.2, frequency=0.1)


def _prompts(seed, lens):
    g = np.random.default_rng(seed)
    return [g.integers(0, 4096, n).tolist() for n in lens]


def _shortfalls(g, model, prompts, texts):
    """How far each token's adjusted logit is below the largest at its place, in spreads of the logits, by whole passes
    of examples/generate.py's decoder and the oracle's penalties."""
    out = []
    allowed = np.arange(g.VOCAB) != 0
    for prompt, text in zip(prompts, texts):
        cache = g.Cache(8, 1, 256)
        logits = g.forward(model, cache, g._int32(prompt), [len(prompt)])
        for i, token in enumerate(text):
            x = logits[0].double().cpu().numpy()
            want, _ = odraft.adjust(x, prompt, text[:i], *PENALTIES.values(), allowed=allowed)
            out.append((want.max() - want[token]) / x.std())
            logits = g.forward(model, cache, g._int32([token]), [1])
    return np.array(out)


def test_rounds_make_the_text_that_the_decoder_chooses():
    import generate as g
    import speculate as sp
    model, prompts, steps = g.Decoder(), _prompts(2, (5, 64, 119)), 14
    first = sp.Rounds(model, prompts, steps, **PENALTIES)
    texts, rounds = first.run()
    assert rounds <= steps and all(len(t) == steps for t in texts)
    # A pass in other shapes differs by 3 % of the logits' spread (root mean square: the sums of attention in another
    # order, each rounded to bf16); two logits, each off by at most five times that, can change their order
    assert _shortfalls(g, model, prompts, texts).max() < 0.3

    # followers that know the text: its tokens are drafted as the last node of each level, and kept in fewer rounds
    follow = sp.followers(model)
    for prompt, text in zip(prompts, texts):
        for a, b in zip(text, text[1:]):
            follow[a, 1] = b
    again = sp.Rounds(model, prompts, steps, follow=follow, **PENALTIES)
    known, fewer = again.run()
    assert _shortfalls(g, model, prompts, known).max() < 0.3
    assert fewer < rounds

    # every sequence ended; a last step takes its pages back
    for r in (first, again):
        assert r.keep.tolist() == [0, 0, 0] and r.fresh.tolist() == [0, 0, 0]
        r.round()
        assert r.held.tolist() == [0, 0, 0] and int(r.state[1]) == len(r.pool)
        assert sorted(r.pool.tolist()) == list(range(len(r.pool)))


def test_a_captured_round_repeats_the_eager_one():
    import generate as g
    import speculate as sp
    model, prompts, steps = g.Decoder(), _prompts(4, (63, 3, 130, 17)), 20
    runs = []
    for eager in (True, False):
        r = sp.Rounds(model, prompts, steps, **PENALTIES)
        texts, rounds = r.run(eager)
        torch.cuda.synchronize()
        runs.append((r, texts, rounds))
    (a, texts, rounds), (b, other, more) = runs
    assert texts == other and rounds == more
    for name in ("pool", "state", "table", "held", "keep", "history", "history_lens", "pending"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    for x, y in zip(a.caches, b.caches):
        assert torch.equal(x.data, y.data)

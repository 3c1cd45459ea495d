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


def _everything(stream=None):
    """Results of one call of each on fixed inputs: a small round without a model."""
    import verify_nvfp4_w4a16_amd as nv
    import workload
    from tests._kv import Paged, bf16, int32, starts
    from tests.test_gpu_draft import _parents
    from tests.test_gpu_kv import _query_bits
    g = workload.rng(8)
    lens, new = [300, 70, 129], [20, 33, 7]
    c = Paged(lens, 2, 128, 77, extra=4)
    total, most = sum(new), max(new)
    parents = int32(np.concatenate([_parents(g, n) for n in new]))
    drafted, chosen = (int32(g.integers(0, 3, total)) for _ in range(2))
    logits = torch.tensor(g.standard_normal((total, 500)).astype(np.float32), device="cuda:0")
    history, said = int32(g.integers(0, 500, (3, 40))), int32([40, 7, 0])
    half = torch.full((3,), 0.5, device="cuda:0")
    q = bf16(_query_bits(total, 8, 128, 78))
    pool, state = int32(c.free + [-1] * 8), int32([0, len(c.free)])
    table, where = c.table_t.clone(), (c.table_t, c.lens_t, starts(new))
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    step = nv.kv_pages(pool, state, table, int32([-(-n // 64) for n in lens]), c.lens_t, int32([3, 60, 0]), 63, stream=stream)
    masks, positions = nv.kv_tree(parents, *where[1:], most, stream=stream)
    out, lse = nv.kv_tree_attention(q, c.cache, *where, masks, positions, most, 320, window=200, stream=stream)
    adjusted = nv.adjust_logits(logits, history, said, q_starts=where[2], repetition=half + 0.7, presence=half, frequency=half,
                                drafted=drafted, masks=masks, stream=stream)
    path, counts, token, kept = nv.tree_accept(drafted, parents, chosen, *where[1:], most, stream=stream)
    nv.kv_move(c.cache, *where, path, stream=stream)
    if stream is not None:
        stream.synchronize()
    torch.cuda.synchronize()
    return (pool, table, *step, masks, positions, out, lse, adjusted, path, counts, token, kept, c.data)


def test_every_call_on_another_stream():
    want = _everything()
    side = torch.cuda.Stream()
    got = _everything(side)
    assert len(want) == len(got)
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(a, b), i


def test_graphs_that_share_a_workspace():
    import verify_nvfp4_w4a16_amd as nv
    import workload
    from tests._kv import DEV, Paged, bf16, starts
    from tests.test_gpu_kv import _query_bits
    from tests.test_gpu_tree_attention import _masks, _of_trees, _wide
    g = workload.rng(9)
    calls, need = [], 0
    for lens, new, wide in (([3000, 100], [16, 12], True), ([2500], [5], False), ([700, 900, 64], [64, 40, 33], True)):
        c = Paged(lens, 1, 128, sum(lens))
        masks, _ = _of_trees(g, lens, new)
        q = bf16(_query_bits(sum(new), 4, 128, sum(new)))
        table, most = _wide(c) if wide else (c.table_t, max(lens))
        args = (q, c.cache, table, c.lens_t, starts(new), _masks(masks, 1), None, max(new), most)
        need = max(need, nv.kv_tree_attention_workspace(c.cache, q, *args[2:5], max(new), most))
        want, want_lse = nv.kv_tree_attention(*args)
        calls.append((args, want, want_lse, torch.empty_like(want), torch.empty_like(want_lse)))
    workspace = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    graphs = []
    for args, _, _, out, lse in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            nv.kv_tree_attention(*args, out=out, lse=lse, workspace=workspace)
    for turn in range(4):
        for i in g.permutation(len(graphs)):
            calls[i][3].zero_()
            calls[i][4].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for _, want, want_lse, out, lse in calls:
            assert torch.equal(out, want) and torch.equal(lse, want_lse), turn

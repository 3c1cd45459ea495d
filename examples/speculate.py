"""Generation in rounds of drafted trees with examples/generate.py's decoder: page
tables on the device, tree attention, penalties, acceptance and its move in the
cache, a whole round in one captured graph (needs an MI355X).

  python examples/speculate.py [--tokens 40] [--eager]

A round drafts, for each sequence, a full tree of two followers a node from a table
(each token's two likeliest followers by the model without its layers), runs the
model once over all nodes, keeps the branch that the model's own choices go along
and moves its slots up.  Nothing in a round waits for the device: page numbers,
lengths and starts never leave it.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from generate import DEV, DIM, HEADS, KV_HEADS, LAYERS, VOCAB, Decoder, norm  # noqa: E402
import verify_nvfp4_w4a16_amd as nv  # noqa: E402

DEPTH = 3
NODES = 2 ** (DEPTH + 1) - 1


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def followers(model):
    """[VOCAB, 2]: each token's two likeliest followers by the embedding and the head alone."""
    logits = torch.cat([model.head(norm(part), torch.float32) for part in model.embed.split(1024)])
    return logits.topk(2, 1).indices


class Rounds:
    """Sequences that grow by drafted trees until each has `steps` new tokens; one that has gives its
    pages back."""

    def __init__(self, model, prompts, steps, follow=None, repetition=1.1, presence=0.2, frequency=0.1):
        self.model, self.steps, n = model, steps, len(prompts)
        self.follow = followers(model) if follow is None else follow
        lens = [len(p) for p in prompts]
        self.most = max(lens) + steps + 2 * NODES
        pitch = -(-self.most // 64)
        pages = n * pitch
        # K and V of a normalised input have a spread near 1: 2^-6 holds up to 42 of it
        self.caches = [nv.KvCache.empty(pages, KV_HEADS, DIM, 2.0 ** -6, 2.0 ** -6, DEV) for _ in range(LAYERS)]
        self.pool, self.state = _int32(np.arange(pages)), _int32([0, pages])
        self.table = torch.full((n, pitch), -1, dtype=torch.int32, device=DEV)
        self.held, self.keep = _int32([0] * n), _int32([0] * n)
        self.fresh = _int32([NODES] * n)
        self.history = torch.zeros((n, max(lens) + steps + DEPTH + 1), dtype=torch.int32, device=DEV)
        for s, p in enumerate(prompts):
            self.history[s, :len(p)] = _int32(p)
        self.prompt_lens, self.history_lens = _int32(lens), _int32(lens)
        full = torch.full((n,), 1.0, device=DEV)
        self.penalties = dict(repetition=full * repetition, presence=full * presence, frequency=full * frequency)
        # token 0 may not come
        self.allowed = torch.full((1, VOCAB // 32), -1, dtype=torch.int32, device=DEV)
        self.allowed[0, 0] = -2
        self.total = n * NODES
        self.no_state = torch.zeros(self.total, dtype=torch.int32, device=DEV)
        self.u = torch.zeros(self.total, device=DEV)
        self.one = torch.ones(self.total, dtype=torch.int32, device=DEV)     # top_k: the likeliest token
        self.shape = _int32([(i - 1) // 2 if i else -1 for i in range(NODES)])
        self.counts = _int32([0] * n)
        self._prompts(lens)

    def _layers(self, tokens, where, attend):
        x = self.model.embed[tokens]
        for layer, cache in zip(self.model.layers, self.caches):
            q, k, v = layer["qkv"](norm(x)).view(-1, HEADS + 2 * KV_HEADS, DIM).split([HEADS, KV_HEADS, KV_HEADS], 1)
            nv.kv_append(cache, k, v, *where)
            x = x + layer["out"](attend(q, cache).view(-1, HEADS * DIM))
            h = norm(x)
            x = x + layer["down"]((torch.nn.functional.silu(layer["gate"](h).float()) * layer["up"](h).float()).bfloat16())
        return x

    def _prompts(self, lens):
        step = nv.kv_pages(self.pool, self.state, self.table, self.held, self.keep, _int32(lens), sum(lens))
        tokens = torch.cat([self.history[s, :n] for s, n in enumerate(lens)])
        where = (self.table, step.kv_lens, step.q_starts)
        x = self._layers(tokens, where, lambda q, c: nv.kv_attention(q, c, *where, max(lens), max(lens))[0])
        logits = self.model.head(norm(x[step.q_starts[1:].long() - 1]), torch.float32)
        logits = nv.adjust_logits(logits, self.history, self.history_lens, prompt_lens=self.prompt_lens, allowed=self.allowed,
                                  allowed_rows=self.no_state[:len(lens)], **self.penalties)
        self.pending, _ = nv.sample(logits, self.u[:len(lens)], top_k=self.one[:len(lens)])
        self.state.copy_(step.state)
        self.held.copy_(step.held)
        self.keep.copy_(step.kv_lens)

    def draft(self, seq, node):
        """Drafted tokens and parents of the packed nodes."""
        level, tree = self.pending[:, None], [self.pending[:, None]]
        for _ in range(DEPTH):
            level = self.follow[level.long()].flatten(1).int()
            tree.append(level)
        return torch.cat(tree, 1)[seq, node].contiguous(), self.shape[node].contiguous()

    def round(self):
        """One round of all sequences; fixed shapes and buffers, so that it can be captured."""
        n = len(self.keep)
        step = nv.kv_pages(self.pool, self.state, self.table, self.held, self.keep, self.fresh, self.total)
        where = (self.table, step.kv_lens, step.q_starts)
        rows = torch.arange(self.total, device=DEV, dtype=torch.int32)
        seq = torch.searchsorted(step.q_starts[1:], rows, right=True).clamp(max=n - 1)
        drafted, parents = self.draft(seq, (rows - step.q_starts[seq]).clamp(0, NODES - 1))
        masks, positions = nv.kv_tree(parents, step.kv_lens, step.q_starts, NODES)
        x = self._layers(drafted, where, lambda q, c: nv.kv_tree_attention(q, c, *where, masks, positions, NODES, self.most)[0])
        # rows behind the last sequence's are no nodes: what they hold is looked at by no call after this one
        logits = nv.adjust_logits(self.model.head(norm(x), torch.float32), self.history, self.history_lens,
                                  prompt_lens=self.prompt_lens, q_starts=step.q_starts, allowed=self.allowed,
                                  allowed_rows=self.no_state, drafted=drafted, masks=masks, **self.penalties)
        chosen, _ = nv.sample(logits, self.u, top_k=self.one)
        path, counts, token, lens = nv.tree_accept(drafted, parents, chosen, step.kv_lens, step.q_starts, NODES)
        nv.kv_move(self.caches, *where, path)

        # the accepted nodes' tokens join the text, and the round's state becomes the next one's
        at = torch.arange(DEPTH + 1, device=DEV)
        taken = drafted[(step.q_starts[:-1, None] + path[:, :DEPTH + 1].clamp(min=0)).clamp(max=self.total - 1).long()]
        place = (self.history_lens[:, None] + at).clamp(max=self.history.shape[1] - 1)
        self.history.scatter_(1, place, torch.where(at < counts[:, None], taken, self.history.gather(1, place)))
        self.history_lens.add_(counts)
        self.counts.copy_(counts)
        done = self.history_lens - self.prompt_lens >= self.steps
        self.pending.copy_(torch.where(counts > 0, token, self.pending))
        self.fresh.copy_(torch.where(done, 0, self.fresh))
        self.keep.copy_(torch.where(done, 0, lens))
        self.held.copy_(step.held)
        self.state.copy_(step.state)

    def run(self, eager=False):
        """(texts, rounds): `steps` new tokens of each sequence and the rounds that they took."""
        rounds = 0
        graph = None
        while bool((self.fresh > 0).any()):
            if eager or rounds == 0:       # the first round also sets up what the library allocates once
                self.round()
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        self.round()
                graph.replay()
            rounds += 1
        return [self.history[s, p:p + self.steps].tolist() for s, p in enumerate(self.prompt_lens.tolist())], rounds


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=40)
    ap.add_argument("--eager", action="store_true", help="call by call instead of a captured graph")
    args = ap.parse_args()
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (5, 70, 119)]
    texts, rounds = Rounds(Decoder(), prompts, args.tokens).run(args.eager)
    for p, t in zip(prompts, texts):
        print(f"prompt of {len(p)} tokens -> {t[:12]} ...")
    print(f"{args.tokens} tokens each in {rounds} rounds")


if __name__ == "__main__":
    main()

"""Generation with a small random decoder: NVFP4 products, the paged NVFP4 cache
and sampling, as a serving loop calls them (needs an MI355X).

  python examples/generate.py [--tokens 40] [--keep 96]

Each layer: QKV product, append, attention over the cache, output product, gated
feed-forward.  A sequence whose cache passes --limit slots is cut to --keep of
them by the attention weight its slots gathered.  Weights are random and there
are no positions: the tokens mean nothing, the calls are the point.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import verify_nvfp4_w4a16_amd as nv  # noqa: E402

DEV = torch.device("cuda:0")
HIDDEN, LAYERS, HEADS, KV_HEADS, DIM, FFN, VOCAB = 1024, 2, 8, 2, 128, 2048, 4096


class Weight:
    """A packed NVFP4 weight [N, K] on the GPU."""

    def __init__(self, rng, n, k):
        packed, scales, self.t = nv.pack((rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32))
        self.n, self.k = n, k
        self.packed, self.scales = torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV)

    def __call__(self, x, dtype=torch.bfloat16):
        """x [M, K] . W^T for any M (the kernel is picked by the row count)."""
        x = x.contiguous()
        y = torch.empty((x.shape[0], self.n), dtype=dtype, device=DEV)
        status = nv.matmul_raw(x.data_ptr(), self.packed.data_ptr(), self.scales.data_ptr(), self.t, y.data_ptr(), x.shape[0], self.n,
                               self.k, nv.OUT_F32 if dtype == torch.float32 else nv.OUT_BF16, torch.cuda.current_stream().cuda_stream)
        if status != nv.OK:
            raise nv.Nvfp4Error(status, "nvfp4_matmul")
        return y


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Decoder:
    def __init__(self, seed=0):
        rng = np.random.default_rng(seed)
        self.embed = torch.from_numpy(rng.standard_normal((VOCAB, HIDDEN)).astype(np.float32)).to(DEV).bfloat16()
        self.layers = [dict(qkv=Weight(rng, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN), out=Weight(rng, HIDDEN, HEADS * DIM),
                            gate=Weight(rng, FFN, HIDDEN), up=Weight(rng, FFN, HIDDEN), down=Weight(rng, HIDDEN, FFN))
                       for _ in range(LAYERS)]
        self.head = Weight(rng, VOCAB, HIDDEN)


class Cache:
    """One page pool a layer, with the sequences' tables: all layers use the same page numbers."""

    def __init__(self, pages, sequences, most):
        # K and V of a normalised input have a spread near 1: 2^-6 holds up to 42 of it
        self.layers = [nv.KvCache.empty(pages, KV_HEADS, DIM, 2.0 ** -6, 2.0 ** -6, DEV) for _ in range(LAYERS)]
        self.free = list(range(pages))
        self.pages = [[] for _ in range(sequences)]
        self.lens = [0] * sequences
        self.weights = torch.zeros(LAYERS, sequences, KV_HEADS, most, device=DEV)   # what each slot gathered
        self.most = most

    def grow(self, new):
        """Room for new[s] tokens of each sequence; returns (table, kv_lens, q_starts) on the GPU."""
        for s, n in enumerate(new):
            self.lens[s] += n
            while len(self.pages[s]) * 64 < self.lens[s]:
                self.pages[s].append(self.free.pop())
        return self.table(self.pages), _int32(self.lens), _int32(np.concatenate([[0], np.cumsum(new)]))

    @staticmethod
    def table(pages):
        width = max(len(p) for p in pages)
        return _int32([p + [-1] * (width - len(p)) for p in pages])

    def cut(self, keep, sink, recent):
        """Every layer's heads cut on their own to `keep` slots, into other pages."""
        target = [[self.free.pop() for _ in range(-(-keep // 64))] for _ in self.pages]
        table, lens = self.table(self.pages), _int32(self.lens)
        for i, layer in enumerate(self.layers):
            _, kept, new_lens = nv.kv_evict(self.weights[i], layer, table, lens, self.table(target), keep, sink=sink, recent=recent)
            self.weights[i].zero_()
            self.weights[i, :, :, :keep] = kept
        for s, pages in enumerate(self.pages):
            self.free += pages
            self.pages[s] = target[s]
        self.lens = new_lens.tolist()


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def forward(model, cache, tokens, new):
    """fp32 logits of each sequence's last new token; tokens are packed, new[s] of sequence s."""
    table, lens, starts = cache.grow(new)
    most_new, most = max(new), max(cache.lens)
    x = model.embed[tokens]
    for i, layer in enumerate(model.layers):
        qkv = layer["qkv"](norm(x)).view(-1, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)               # views: the calls take them as they are
        nv.kv_append(cache.layers[i], k, v, table, lens, starts)
        out, lse = nv.kv_attention(q, cache.layers[i], table, lens, starts, most_new, most)
        got = cache.weights[i][:, :, :most].contiguous()
        cache.weights[i][:, :, :most] = nv.kv_weights(q, lse, cache.layers[i], table, lens, starts, most_new, most, prior=got)
        x = x + layer["out"](out.view(-1, HEADS * DIM))
        h = norm(x)
        x = x + layer["down"]((torch.nn.functional.silu(layer["gate"](h).float()) * layer["up"](h).float()).bfloat16())
    return model.head(norm(x[starts[1:].long() - 1]), torch.float32)


def generate(prompts, steps, keep, limit, seed=0, temperature=0.8, top_k=100, top_p=0.95):
    """Token lists that continue the prompts (lists of token numbers), and the cache."""
    model, n = Decoder(), len(prompts)
    most = max(max(len(p) for p in prompts) + steps, limit + 1)
    cache = Cache(pages=n * (2 * (-(-most // 64)) + 2), sequences=n, most=most)
    uniform = torch.Generator(device=DEV).manual_seed(seed)
    params = [torch.full((n,), v, dtype=d, device=DEV) for v, d in ((temperature, torch.float32), (top_k, torch.int32), (top_p, torch.float32))]
    tokens, new = _int32(np.concatenate(prompts)), [len(p) for p in prompts]
    made = []
    for _ in range(steps):
        logits = forward(model, cache, tokens, new)
        tokens, _ = nv.sample(logits, torch.rand(n, generator=uniform, device=DEV), *params)
        new = [1] * n
        made.append(tokens)
        if max(cache.lens) > limit:
            cache.cut(keep, sink=4, recent=keep // 4)
    return torch.stack(made, 1).tolist(), cache


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=40)
    ap.add_argument("--keep", type=int, default=96)
    ap.add_argument("--limit", type=int, default=128)
    args = ap.parse_args()
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (5, 70, 119)]
    texts, cache = generate(prompts, args.tokens, args.keep, args.limit)
    for p, t in zip(prompts, texts):
        print(f"prompt of {len(p)} tokens -> {t[:12]} ...")
    print("cache lengths:", cache.lens)


if __name__ == "__main__":
    main()

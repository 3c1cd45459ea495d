"""Paged caches for the serving tests, built byte by byte from random codes with
the oracle's layout, and kept on both sides.  Not a test module."""
from __future__ import annotations

import numpy as np
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle import kv as okv

DEV = torch.device("cuda:0")
PAGE = okv.PAGE


def int32(a) -> torch.Tensor:
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def bf16(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(DEV).view(torch.bfloat16)


class Paged:
    """Sequences of the given lengths in shuffled pages of one cache; slots beyond a length hold
    bytes of 0xFF (a NaN scale), and `extra` spare pages are free."""

    def __init__(self, lens, heads, d, seed, extra=0, k_scale=2.0 ** -5, v_scale=3e-3):
        g = workload.rng(seed)
        self.lens, self.heads, self.d = list(lens), heads, d
        self.k_scale, self.v_scale = float(np.float32(k_scale)), float(np.float32(v_scale))
        need = [-(-n // PAGE) for n in self.lens]
        pages = sum(need) + extra
        order = g.permutation(pages).tolist()
        self.table = np.full((len(self.lens), max(need + [1])), -1, np.int32)
        data = np.full((max(pages, 1), heads, 72 * d), 0xFF, np.uint8)
        self.k, self.v = [], []                       # [seq][head] float64 [len, D]
        at = 0
        for s, n in enumerate(self.lens):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            ks, vs = [np.zeros((heads, n, d)) for _ in range(2)]
            for h in range(heads):
                rows = need[s] * PAGE
                codes = g.integers(0, 16, (2, rows, d), dtype=np.uint8)
                # scales around 1, so that scores spread over a few units, with the ends of the range among them
                scales = g.integers(0x28, 0x40, (2, rows, d // 16), dtype=np.uint8)
                scales[1][g.random(scales[1].shape) < 0.02] = 0x7E
                scales[0][g.random(scales[0].shape) < 0.02] = 0x01
                scales[:, n:] = 0xFF
                codes[:, n:] = 0xF
                for p in range(need[s]):
                    i = slice(p * PAGE, (p + 1) * PAGE)
                    data[self.table[s, p], h] = okv.build_record(codes[0, i], scales[0, i], codes[1, i], scales[1, i])
                ks[h] = okv.values(codes[0, :n], scales[0, :n], self.k_scale) if n else ks[h]
                vs[h] = okv.values(codes[1, :n], scales[1, :n], self.v_scale) if n else vs[h]
            self.k.append(ks)
            self.v.append(vs)
        self.free = order[at:]
        self.data = torch.from_numpy(data).to(DEV)
        self.cache = nv.KvCache(self.data, heads, d, self.k_scale, self.v_scale)
        self.table_t = int32(self.table)
        self.lens_t = int32(self.lens)


def starts(new) -> torch.Tensor:
    return int32(np.concatenate([[0], np.cumsum(new)]))


def stored(data: np.ndarray, table, n: int, head: int, d: int):
    """(K codes, K scales, V codes, V scales) of a sequence's first n slots, from the cache's bytes."""
    parts = [okv.split_record(data[p, head], d) for p in table[:-(-n // PAGE)]]
    return [np.concatenate([p[i] for p in parts])[:n] for i in range(4)]

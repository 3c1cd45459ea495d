"""Reference of the verify round over drafted trees, from the rules of
include/nvfp4_draft.h: Python integers for tables, trees and branches, float64
for attention and logits.  Loops over sequences, nodes and slots.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def pages(pool, state, table, held, keep, fresh, total):
    """(pool, state, table, held, kv_lens, q_starts, slots, positions) after a step."""
    pool, table = [int(x) for x in pool], np.array(table, np.int64)
    cap, pitch = len(pool), table.shape[1]
    head, count = int(state[0]) % cap, min(max(int(state[1]), 0), cap)   # Python's remainder is not negative
    taken, back = 0, []
    asked = wanted_pages = 0
    out_held, lens, starts, slots, positions = [], [], [0], [], []
    for s in range(len(held)):
        h = min(max(int(held[s]), 0), pitch)
        k = min(max(int(keep[s]), 0), PAGE * h)
        f = max(int(fresh[s]), 0)
        need = -(-(k + f) // PAGE)
        granted = need <= pitch
        if granted:
            asked += f
            wanted_pages += max(need - h, 0)
            granted = (need <= h or wanted_pages <= count) and (f == 0 or asked <= total)
        if not granted:
            f, need = 0, h
        for p in range(h, need):
            table[s, p] = pool[(head + taken) % cap]
            taken += 1
        back += [int(table[s, p]) for p in range(need, h)]
        out_held.append(need)
        lens.append(k + f)
        starts.append(starts[-1] + f)
        for j in range(k, k + f):
            page = int(table[s, j // PAGE])
            slots.append(page * PAGE + j % PAGE if 0 <= page < 1 << 25 else -1)
            positions.append(j)
    back = back[:cap - count]
    for i, p in enumerate(back):
        pool[(head + count + i) % cap] = p
    rest = [-1] * (total - len(slots))
    return (pool, [(head + taken) % cap, count - taken + len(back)], table, out_held, lens, starts, slots + rest, positions + rest)


def ways(parents) -> list[list[int]]:
    """For each node of one tree the nodes from its root to itself."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def mask_words(way, words: int) -> list[int]:
    bits = sum(1 << a for a in way)
    return [(bits >> 64 * w) & (2 ** 64 - 1) for w in range(words)]


def visible(n: int, masks, positions, window: int, whole_tree: bool = False) -> np.ndarray:
    """[nq, n]: which slots each node sees.  masks: a Python integer of bits a node."""
    nq = len(masks)
    before = n - nq
    seen = np.zeros((nq, n), bool)
    place = [min(max(int(p), before), n - 1) for p in positions] if positions is not None else [0] * nq
    for i in range(nq):
        for j in range(max(before, 0)):
            seen[i, j] = not window or j > place[i] - window
        for a in range(nq):
            if masks[i] >> a & 1 and before + a >= 0:
                seen[i, before + a] = not window or whole_tree or place[a] > place[i] - window
    return seen


def attention(q, k, v, seen, scale, softcap=0.0):
    """(out [nq, D], lse [nq], spread [nq, D] = sum p |v|, size [nq]: the largest sum of magnitudes behind a score) of one query head."""
    z = scale * (q @ k.T)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    if softcap:
        z = softcap * np.tanh(z / softcap)
    out, spread = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1]))
    lse, largest = np.full(len(q), -np.inf), np.zeros(len(q))
    for i, m in enumerate(seen):
        if not m.any():
            continue
        top = z[i, m].max()
        e = np.exp(z[i, m] - top)
        out[i], spread[i] = e @ v[m] / e.sum(), e @ np.abs(v[m]) / e.sum()
        lse[i] = top + np.log(e.sum())
        largest[i] = size[i, m].max()
    return out, lse, spread, largest


def adjust(x, prompt, said, r=1.0, p=0.0, f=0.0, bias=(), allowed=None):
    """(adjusted float64 logits, sum of the magnitudes that were rounded on the way) of one row.
    prompt, said: token lists; bias: (token, value) pairs; allowed: truth values."""
    x = np.array(x, np.float64)
    size = np.zeros_like(x)
    r = r if r > 0 else 1.0
    n = np.bincount(np.array([t for t in said if 0 <= t < len(x)], np.int64), minlength=len(x))
    asked = np.bincount(np.array([t for t in prompt if 0 <= t < len(x)], np.int64), minlength=len(x))
    with np.errstate(invalid="ignore", over="ignore"):
        if r != 1.0:
            x = np.where((n > 0) | (asked > 0), np.where(x > 0, x / r, x * r), x)
            size += np.abs(x)
        if p or f:
            size += np.where(n > 0, np.abs(x - p) + np.abs(f * n), 0.0)
            x = np.where(n > 0, x - p - f * n, x)
            size += np.where(n > 0, np.abs(x), 0.0)
        for t, value in dict((t, value) for t, value in bias).items():
            if 0 <= t < len(x):
                x[t] += value
                size[t] += abs(x[t])
    if allowed is not None:
        x = np.where(allowed, x, -np.inf)
    return x, size


def accept(drafted, parents, chosen):
    """(path, token) of one tree."""
    if not len(drafted):
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        after = [c for c in range(at + 1, len(drafted)) if parents[c] == at and drafted[c] == chosen[at] and drafted[c] >= 0]
        if not after:
            return path, int(chosen[at])
        path.append(after[0])

"""Reference of the token choice: exact integer masses in Python integers.

The weights floor(2^30 exp d) take the exponential in float64, the library in
fp32, so `margin` says how far (relative to the masses compared) the nearest
decision was from falling otherwise; a caller compares tokens only where it is
well above fp32's error of the exponential.
"""
from __future__ import annotations

import numpy as np

STEPS = 1 << 30


def sample(logits: np.ndarray, u: float, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, margin) of one row of fp32 logits."""
    x = np.where(np.isnan(logits), -np.inf, logits).astype(np.float32)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf, np.inf
    margin = np.inf
    if temperature > 0:
        inverse = np.float32(1.0) / np.float32(temperature)
        with np.errstate(invalid="ignore"):
            d = ((x - top) * inverse).astype(np.float64)
        w = np.where(x == top, STEPS, np.floor(np.exp(np.where(x == top, 0.0, d)) * STEPS)).astype(np.int64)
    else:
        w = np.where(x == top, STEPS, 0).astype(np.int64)
        top_k = 1
    order = sorted((i for i in range(len(w)) if w[i] > 0), key=lambda i: (-w[i], i))
    if 0 < top_k < len(order):
        a, b = int(w[order[top_k - 1]]), int(w[order[top_k]])
        if x[order[top_k - 1]] != x[order[top_k]]:
            margin = min(margin, (a - b) / a)
        order = order[:top_k]
    mass = sum(int(w[i]) for i in order)
    kept, before = [], 0
    limit = float(np.float32(top_p)) * float(mass)
    low = float(np.float32(min_p)) * STEPS
    for place, i in enumerate(order):
        wi = int(w[i])
        if top_p < 1:
            margin = min(margin, abs(before - limit) / mass)
        if min_p > 0 and place:
            margin = min(margin, abs(wi - low) / low)
        if place == 0 or (before < limit and wi >= low):
            kept.append(i)
        before += wi
    total = sum(int(w[i]) for i in kept)
    target = min(int(float(np.float32(u)) * float(total)), total - 1)
    run = 0
    for i in sorted(kept):
        margin = min(margin, abs(run - target) / total) if run else margin
        run += int(w[i])
        if run > target:
            margin = min(margin, (run - target) / total) if i != max(kept) else margin
            return i, float(np.log(int(w[i]) / total)), margin
    raise AssertionError("the running mass ends above every target")

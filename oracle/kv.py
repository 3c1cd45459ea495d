"""Float64 reference of the paged NVFP4 key/value cache and what reads it.

Written from the rules of include/nvfp4_kv.h: a record's layout byte by byte,
attention, the weight of slots, eviction.  Everything works on one sequence and
one kv head at a time.
"""
from __future__ import annotations

import numpy as np

from .formats import E2M1, E4M3
from .linear import bf16_bits_to_f64
from .quant import e2m1_round, e4m3_round

PAGE = 64


def k_scale_index(slot: int, group: int, d: int) -> int:
    """Byte of K's scale of (slot, 16-dim group) within a record."""
    h, a, t, r = slot // 32, slot // 8 % 4, slot // 4 % 2, slot % 4
    per = d // 64
    return 64 * d + ((((a * 4 + r) * 4 + group // per) * 2 + h) * 2 + t) * per + group % per


def v_scale_index(slot: int, group: int, d: int) -> int:
    return 68 * d + (slot // 8 * (d // 16) + group) * 8 + slot % 8


def build_record(k_codes, k_scales, v_codes, v_scales) -> np.ndarray:
    """A record (72 D bytes) of codes [64, D] (0..15) and scale bytes [64, D/16]."""
    d = k_codes.shape[1]
    rec = np.zeros(72 * d, np.uint8)
    rec[:32 * d] = (k_codes[:, 0::2] | (k_codes[:, 1::2] << 4)).reshape(-1)
    for block in range(8):
        c = v_codes[8 * block:8 * block + 8]                     # [8, D]
        dwords = (c[0::2] | (c[1::2] << 4)).T                    # [D, 4]
        rec[32 * d + block * d * 4:32 * d + (block + 1) * d * 4] = dwords.reshape(-1)
    for slot in range(PAGE):
        for g in range(d // 16):
            rec[k_scale_index(slot, g, d)] = k_scales[slot, g]
            rec[v_scale_index(slot, g, d)] = v_scales[slot, g]
    return rec


def split_record(rec: np.ndarray, d: int):
    """The inverse of build_record."""
    kb = rec[:32 * d].reshape(PAGE, d // 2)
    k = np.stack([kb & 15, kb >> 4], -1).reshape(PAGE, d)
    vb = rec[32 * d:64 * d].reshape(8, d, 4)
    v = np.stack([vb & 15, vb >> 4], -1).reshape(8, d, 8).transpose(0, 2, 1).reshape(PAGE, d)
    ks = np.array([[rec[k_scale_index(s, g, d)] for g in range(d // 16)] for s in range(PAGE)], np.uint8)
    vs = np.array([[rec[v_scale_index(s, g, d)] for g in range(d // 16)] for s in range(PAGE)], np.uint8)
    return k, ks, v, vs


def values(codes, scales, t: float) -> np.ndarray:
    """[rows, D] float64 values of codes and scale bytes."""
    return t * E2M1[codes] * np.repeat(E4M3[scales], 16, axis=1)


def quantise_rows(bits: np.ndarray, t: float):
    """(codes, scale bytes) of bf16 rows [rows, D] at the tensor scale t: nvfp4_pack's rule,
    a NaN counting as 0 and an infinity saturating."""
    x = bf16_bits_to_f64(bits)
    x = np.where(np.isnan(x), 0.0, x)
    rows, d = x.shape
    g = x.reshape(rows, d // 16, 16)
    u = np.abs(g).max(-1) / 6.0 / np.float64(np.float32(t))
    scales = e4m3_round(np.minimum(u, 1e300))
    big = (E4M3[scales] * np.float64(np.float32(t)))[..., None]
    codes = e2m1_round(np.clip(g / np.where(big > 0, big, 1.0), -1e300, 1e300))
    codes[np.broadcast_to(big, g.shape) == 0.0] = 0
    return codes.reshape(rows, d), scales


def visible(n: int, nq: int, causal: bool, window: int) -> np.ndarray:
    """[nq, n] truth values: which slots each new token sees."""
    p = n - nq + np.arange(nq)[:, None]
    j = np.arange(n)[None]
    seen = np.ones((nq, n), bool)
    if causal:
        seen &= j <= p
    if window:
        seen &= j > p - window
    return seen


def scores(q, k, scale: float, softcap: float):
    """(scores [nq, n], sum of magnitudes behind each) of q [nq, D] and k [n, D]."""
    z = scale * (q @ k.T)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    if softcap:
        z = softcap * np.tanh(z / softcap)
    return z, size


def attention(q, k, v, scale, causal=True, window=0, softcap=0.0):
    """(out [nq, D], lse [nq], spread [nq, D] = sum p |v|, size [nq]) of one query head."""
    nq, n = q.shape[0], k.shape[0]
    z, size = scores(q, k, scale, softcap)
    seen = visible(n, nq, causal, window)
    out, lse = np.zeros((nq, v.shape[1])), np.full(nq, -np.inf)
    spread, largest = np.zeros_like(out), np.zeros(nq)
    for i in range(nq):
        m = seen[i]
        if not m.any():
            continue
        top = z[i, m].max()
        e = np.exp(z[i, m] - top)
        out[i] = e @ v[m] / e.sum()
        spread[i] = e @ np.abs(v[m]) / e.sum()
        lse[i] = top + np.log(e.sum())
        largest[i] = size[i, m].max()
    return out, lse, spread, largest


def slot_weights(q, k, lse, scale, causal=True, window=0, softcap=0.0):
    """(weights [n], size [n]: each slot's weights times the magnitudes behind their scores) of one head."""
    nq, n = q.shape[0], k.shape[0]
    z, size = scores(q, k, scale, softcap)
    seen = visible(n, nq, causal, window) & np.isfinite(lse)[:, None]
    p = np.where(seen, np.exp(np.where(seen, z, 0.0) - np.where(np.isfinite(lse), lse, 0.0)[:, None]), 0.0)
    return p.sum(0), (p * size).sum(0)


def evict(weights, n: int, keep: int, sink: int, recent: int) -> np.ndarray:
    """Slots that stay, ascending."""
    if n <= keep:
        return np.arange(n)
    w = np.where(np.isnan(weights[:n]), -np.inf, weights[:n]).astype(np.float64)
    middle = sorted(range(sink, n - recent), key=lambda j: (-w[j], j))[:keep - sink - recent]
    return np.array(sorted(list(range(sink)) + middle + list(range(n - recent, n))))

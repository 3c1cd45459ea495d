"""The paged NVFP4 cache on the GPU (gpu): append, read, attention, slot
weights and eviction against the float64 oracle, at the lengths, masks, strides
and head counts where they can go wrong.

Tolerances.  A score is a D-term fp32 sum of exact products (its error at most
(D + 8) 2^-24 times the sum of magnitudes `size`, the scalings by powers of two
and one or two roundings included; the tanh form adds a few rounding errors of
a value at most the cap), so exp(z - m) is off by a relative
eps = 2 (D + 8) 2^-24 size + 2^-20 at most.  The attention weights are rounded
to f16 (2^-11, and 2^-25 absolute below f16's normal range), and the output to
bf16 (8 significant bits: 2^-8): |out - ref| <= 2^-8 |ref| + (eps + 2^-10) sum p|v| + n 2^-24 max|v|."""
import numpy as np
import pytest
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle import kv as okv
from oracle import bf16_bits_to_f64
from tests._kv import DEV, PAGE, Paged, bf16, int32, starts, stored

pytestmark = pytest.mark.gpu


def _eps(size, d, softcap):
    return 2 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20 + (8 * softcap * 2.0 ** -23)


def _query_bits(total, heads, d, seed):
    return workload.activations_bf16(total, heads * d, seed).reshape(total, heads, d)


def _attend(c, qbits, new, strided=False, max_q=None, max_kv=None, **kw):
    q = bf16(qbits)
    if strided:                                              # a view of a fused projection's output
        total, heads, d = q.shape
        wide = torch.full((total, heads * d + 2 * c.heads * d), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :heads * d] = q.reshape(total, heads * d)
        q = wide[:, :heads * d].view(total, heads, d)
    out, lse = nv.kv_attention(q, c.cache, c.table_t, c.lens_t, starts(new), max_q or max(max(new), 1),
                               max_kv if max_kv is not None else max(max(c.lens), 1), **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def _check(c, qbits, new, out, lse, causal=True, window=0, softcap=0.0, scale=None):
    q = bf16_bits_to_f64(qbits)
    heads, d = q.shape[1], c.d
    scale = d ** -0.5 if scale is None else scale
    group = heads // c.heads
    at, worst = 0, 0.0
    for s, n in enumerate(c.lens):
        for h in range(heads):
            k, v = c.k[s][h // group], c.v[s][h // group]
            o, l, spread, size = okv.attention(q[at:at + new[s], h], k, v, scale, causal, window, softcap)
            eps = _eps(size, d, softcap)[:, None]
            top = np.abs(v).max() if n else 0.0
            tol = 2.0 ** -8 * np.abs(o) + (eps + 2.0 ** -10) * spread + (n + 1) * 2.0 ** -24 * top
            err = np.abs(out[at:at + new[s], h] - o)
            assert np.all(err <= tol), (s, h, float((err / np.maximum(tol, 1e-300)).max()))
            got = lse[at:at + new[s], h]
            empty = ~np.isfinite(l)
            assert np.array_equal(np.isneginf(got), empty), (s, h)
            assert np.all(out[at:at + new[s], h][empty] == 0.0)
            lim = eps[:, 0] + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(empty, 0, l)))
            assert np.all(np.abs(got - l)[~empty] <= lim[~empty]), (s, h, np.abs(got - l)[~empty].max())
        at += new[s]


CASES = [
    # lens, new, kv heads, group, D, options
    ([1], [1], 1, 1, 64, {}),
    ([1, 2, 63, 64, 65], [1, 1, 1, 1, 1], 2, 4, 128, {}),
    ([700, 5, 129], [1, 1, 1], 2, 7, 64, {}),
    ([300, 31, 16], [1, 1, 1], 1, 16, 256, {}),
    ([130, 77], [5, 7], 2, 3, 128, {}),
    ([130, 77], [5, 7], 2, 3, 128, dict(causal=False)),
    ([130, 200, 64], [17, 33, 64], 1, 2, 64, {}),
    ([200, 131], [70, 131], 2, 4, 128, {}),
    ([200, 131], [40, 90], 1, 5, 256, {}),
    ([333, 64, 65, 1], [9, 2, 64, 1], 2, 2, 128, dict(window=1)),
    ([333, 64, 65, 1], [9, 2, 64, 1], 2, 2, 128, dict(window=67)),
    ([333, 70], [1, 1], 2, 8, 64, dict(window=64)),
    ([333, 70], [1, 30], 2, 1, 256, dict(window=100, softcap=5.0)),
    ([150, 260], [150, 3], 1, 8, 128, dict(softcap=30.0)),
    ([90, 260], [4, 1], 1, 32, 128, dict(causal=False, window=80)),
    ([0, 5, 0], [1, 1, 0], 1, 2, 64, {}),                      # nothing cached: empty rows
    ([3, 2], [8, 5], 1, 2, 64, {}),                            # more new tokens than slots: the first see nothing
    ([500, 40], [0, 3], 2, 2, 128, {}),                        # a sequence without new tokens
]


@pytest.mark.parametrize("lens,new,heads,group,d,kw", CASES)
def test_attention(lens, new, heads, group, d, kw):
    c = Paged(lens, heads, d, 100 + sum(lens))
    qb = _query_bits(sum(new), heads * group, d, 7 + d)
    out, lse = _attend(c, qb, new, strided=len(lens) % 2 == 0, **kw)
    _check(c, qb, new, out, lse, **kw)


# 33 to 64 rows a kv head, which one workgroup takes with the page's halves apart
@pytest.mark.parametrize("lens,new,heads,group,d,kw", [
    ([333, 64, 65, 1], [9, 2, 16, 1], 2, 4, 128, {}),
    ([100, 31], [16, 11], 1, 4, 64, dict(window=40)),
    ([200, 33, 0], [5, 7, 0], 1, 9, 256, dict(softcap=8.0)),
    ([5000, 40], [16, 3], 1, 4, 128, {}),
    ([3000, 40], [33, 3], 2, 1, 256, dict(causal=False, window=2000)),
    ([20, 3], [33, 5], 1, 1, 64, {}),
])
def test_attention_of_a_verify_round(lens, new, heads, group, d, kw):
    c = Paged(lens, heads, d, 300 + sum(lens))
    qb = _query_bits(sum(new), heads * group, d, 17 + d)
    out, lse = _attend(c, qb, new, **kw)
    _check(c, qb, new, out, lse, **kw)
    again = _attend(c, qb, new, **kw)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


def test_attention_with_a_negative_scale():
    for new, lens in (([1, 1], [200, 70]), ([40, 3], [200, 70])):
        c = Paged(lens, 1, 128, 23)
        qb = _query_bits(sum(new), 4, 128, 24)
        out, lse = _attend(c, qb, new, scale=-0.2)
        _check(c, qb, new, out, lse, scale=-0.2)


def test_attention_of_many_sequences_of_very_different_lengths():
    # enough workgroups' worth of bound that the pages are planned from the lengths; empty ones among them
    g = workload.rng(31)
    lens = [int(x) for x in np.exp(g.uniform(0, np.log(2500), 70))]
    lens[3], lens[40], lens[-1] = 0, 12000, 1
    new = [min(1, n) for n in lens]
    c = Paged(lens, 4, 64, 32)
    qb = _query_bits(sum(new), 8, 64, 33)
    out, lse = _attend(c, qb, new)
    _check(c, qb, new, out, lse)
    again = _attend(c, qb, new)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("d,new,group", [(64, 1, 4), (128, 1, 4), (128, 40, 4), (256, 20, 2)])
def test_attention_over_many_splits_repeats_its_bits(d, new, group):
    lens = [5000, 1, 2049]
    c = Paged(lens, 1, d, 33)
    news = [new, 1, min(new, 2049)]
    qb = _query_bits(sum(news), group, d, 9)
    first = _attend(c, qb, news)
    _check(c, qb, news, *first)
    for _ in range(3):
        again = _attend(c, qb, news)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_attention_bounds_that_exceed_the_lengths():
    lens, new = [100, 9], [3, 1]
    c = Paged(lens, 2, 128, 5)
    qb = _query_bits(4, 4, 128, 6)
    out, lse = _attend(c, qb, new, max_q=50, max_kv=c.table.shape[1] * PAGE)
    _check(c, qb, new, out, lse)


def test_attention_of_large_and_small_queries():
    # bf16 reaches beyond f16 at both ends; a row's own power of two brings it back
    c = Paged([90], 1, 128, 8)
    qb = _query_bits(6, 2, 128, 9)
    q = workload.bf16_bits_to_f32(qb)
    q[0] *= 2.0 ** 60
    q[1] *= 2.0 ** -90
    q[2, 0] = 0.0
    q[3, :, ::2] *= 2.0 ** -30
    qb = workload.f32_to_bf16_bits(q)
    for scale in (128 ** -0.5,):
        out, lse = _attend(c, qb[1:], [5], scale=scale)
        _check(c, qb[1:], [5], out, lse, scale=scale)
    out, lse = _attend(c, qb[:1], [1], scale=2.0 ** -62)
    _check(c, qb[:1], [1], out, lse, scale=2.0 ** -62)


def test_attention_nan_and_infinite_queries_stay_in_their_rows():
    c = Paged([150], 1, 64, 8)
    qb = _query_bits(5, 3, 64, 9)
    clean = _attend(c, qb, [5])
    bad = qb.copy()
    bad[1, 1, 3] = 0x7FC0          # NaN
    bad[3, 2, 0] = 0x7F80          # inf
    out, lse = _attend(c, bad, [5])
    hit = np.zeros((5, 3), bool)
    hit[1, 1] = hit[3, 2] = True
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert np.array_equal(out[~hit], clean[0][~hit]) and np.array_equal(lse[~hit], clean[1][~hit])


def test_attention_skips_pages_outside_the_cache():
    # a page number that the cache does not have stands for slots that nothing sees
    c = Paged([200, 90], 1, 64, 12)
    qb = _query_bits(2, 2, 64, 3)
    table = c.table.copy()
    table[0, 1] = 10 ** 6
    table[1, 0] = -7
    c.table_t = int32(table)
    out, lse = _attend(c, qb, [1, 1])
    keep = [np.r_[0:64, 128:200], np.r_[64:90]]
    for s in range(2):
        c.k[s], c.v[s] = c.k[s][:, keep[s]], c.v[s][:, keep[s]]
    c.lens = [len(k) for k in keep]
    _check(c, qb, [1, 1], out, lse)


def test_attention_on_another_stream_and_in_a_graph():
    c = Paged([700, 64], 2, 128, 21)
    new = [1, 1]
    qb = _query_bits(2, 8, 128, 22)
    want, want_lse = _attend(c, qb, new)
    q, st = bf16(qb), starts(new)
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((2, 8), dtype=torch.float32, device=DEV)
    ws = torch.empty(nv.kv_attention_workspace(c.cache, q, c.table_t, c.lens_t, st, 1, 700), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nv.kv_attention(q, c.cache, c.table_t, c.lens_t, st, 1, 700, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert np.array_equal(out.float().cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv_attention(q, c.cache, c.table_t, c.lens_t, st, 1, 700, out=out, lse=lse, workspace=ws)
    for _ in range(4):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy(), want) and np.array_equal(lse.cpu().numpy(), want_lse)


@pytest.mark.parametrize("lens,new,heads,d", [([1], [1], 1, 64), ([64, 65, 130], [64, 1, 70], 2, 128),
                                              ([9, 200, 31], [3, 11, 31], 1, 256), ([5, 100], [0, 9], 3, 64),
                                              ([3], [5], 1, 64)])
def test_append_and_read(lens, new, heads, d):
    c = Paged(lens, heads, d, 40 + d, v_scale=2.7e-3)
    before = c.data.cpu().numpy().copy()
    g = workload.rng(41)
    x = (g.standard_normal((sum(new), 2 * heads, d)) * np.exp(g.uniform(-6, 1, (sum(new), 2 * heads, 1)))).astype(np.float32)
    x[0, 0, :16] = 0.0                                        # a zero group
    x[-1, -1, :16] = 1e30                                     # saturates the scale
    x[0, 0, 16:32] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * 2.0 ** -5   # ties
    if sum(new) > 1:
        x[1, heads, 16:20] = [np.nan, np.inf, -np.inf, 1.0]
    bits = workload.f32_to_bf16_bits(x)
    rows = bf16(bits)
    nv.kv_append(c.cache, rows[:, :heads], rows[:, heads:], c.table_t, c.lens_t, starts(new))
    ko, vo = nv.kv_read(c.cache, c.table_t, c.lens_t, starts(new), sum(new))
    torch.cuda.synchronize()
    after = c.data.cpu().numpy()
    at = 0
    for s, n in enumerate(lens):
        drop = max(0, new[s] - n)                             # rows before slot 0
        for h in range(heads):
            old = stored(before, c.table[s], n, h, d)
            got = stored(after, c.table[s], n, h, d)
            kept = n - (new[s] - drop)
            for a, b in zip(old, got):
                assert np.array_equal(a[:kept], b[:kept])     # slots before the new ones keep their bytes
            for which, (col, t, out) in enumerate(((h, c.k_scale, ko), (heads + h, c.v_scale, vo))):
                codes, scales = okv.quantise_rows(bits[at + drop:at + new[s], col], t)
                assert np.array_equal(got[2 * which][kept:], codes), (s, h, which)
                assert np.array_equal(got[2 * which + 1][kept:], scales), (s, h, which)
                # the fp32 product rounded to bf16: t * (e4m3 * e2m1), the parenthesis exact
                val = okv.values(codes, scales, 1.0).astype(np.float32) * np.float32(t)
                want = workload.f32_to_bf16_bits(val)
                read = out[at:at + new[s], h].view(torch.int16).cpu().numpy().view(np.uint16)
                assert np.array_equal(workload.bf16_bits_to_f32(read[drop:]), workload.bf16_bits_to_f32(want))
                assert not read[:drop].any()
        at += new[s]
    # every page that holds no sequence's slots, and every slot after the lengths, kept its bytes
    for s, n in enumerate(lens):
        full = len([p for p in c.table[s] if p >= 0]) * PAGE
        for h in range(heads):
            for a, b in zip(stored(before, c.table[s], full, h, d), stored(after, c.table[s], full, h, d)):
                assert np.array_equal(a[n:], b[n:])


@pytest.mark.parametrize("t", [2.0 ** -7, 1.2421875 * 2.0 ** -5, 1.001953125 * 2.0 ** -4, 2.7e-3, 1.0 / 3.0, 2.0 ** -59, 2.0 ** 59,
                               2.0 ** -61, 3.3e-21, 7.7e20, 2.0 ** -110])
def test_append_codes_at_and_beside_the_boundaries(t):
    """Every boundary between two codes, its bf16 neighbours on both sides, at tensor scales of
    few and of many bits, within and beyond the range in which quotients are formed in fp32."""
    d, heads, n = 128, 1, 192
    t = float(np.float32(t))
    g = workload.rng(90)
    bounds = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
    s = np.array([0x08, 0x1F, 0x2D, 0x38, 0x3B, 0x47, 0x7E, 0x03])[g.integers(0, 8, (n, d // 16))]
    big = okv.E4M3[s] * t
    x = bounds[g.integers(0, 7, (n, d // 16, 16))] * big[..., None]
    x[..., 0] = 6.0 * big                                     # the scale comes out as s, nearly always
    bits = workload.f32_to_bf16_bits(np.clip(x, 0, 3e38).astype(np.float32)).astype(np.int64)
    bits[..., 1:] = np.clip(bits[..., 1:] + g.integers(-1, 2, bits[..., 1:].shape), 0, 0x7F7F)
    bits |= g.integers(0, 2, bits.shape) << 15
    bits = bits.reshape(n, heads, d).astype(np.uint16)
    cache = nv.KvCache.empty(3, heads, d, t, t)
    rows = bf16(bits)
    nv.kv_append(cache, rows, rows, int32([[2, 0, 1]]), int32([n]), int32([0, n]))
    torch.cuda.synchronize()
    codes, scales = okv.quantise_rows(bits[:, 0], t)
    got = stored(cache.data.cpu().numpy(), [2, 0, 1], n, 0, d)
    for which in (0, 2):
        assert np.array_equal(got[which + 1], scales)
        assert np.array_equal(got[which], codes)


def test_append_one_by_one_equals_append_at_once():
    d, heads, n = 128, 2, 75
    bits = workload.activations_bf16(n, 2 * heads * d, 50).reshape(n, 2 * heads, d)
    rows = bf16(bits)
    a, b = (nv.KvCache.empty(2, heads, d, 2.0 ** -6, 2.0 ** -6) for _ in range(2))
    table = int32([[1, 0]])
    nv.kv_append(a, rows[:, :heads], rows[:, heads:], table, int32([n]), int32([0, n]))
    for i in range(n):
        nv.kv_append(b, rows[i:i + 1, :heads], rows[i:i + 1, heads:], table, int32([i + 1]), int32([0, 1]))
    torch.cuda.synchronize()
    assert torch.equal(a.data, b.data)


@pytest.mark.parametrize("lens,new,heads,group,d,kw", [
    ([1, 70], [1, 1], 1, 1, 64, {}),
    ([200, 64, 333], [1, 1, 1], 2, 4, 128, {}),
    ([200, 64, 333], [33, 20, 7], 2, 3, 128, {}),
    ([150, 90], [90, 90], 1, 5, 64, dict(window=50)),
    ([300, 40], [5, 2], 1, 9, 256, dict(softcap=10.0)),
    ([130, 40], [12, 40], 1, 2, 128, dict(causal=False, window=30)),
    ([0, 3], [2, 5], 1, 2, 64, {}),
])
def test_slot_weights(lens, new, heads, group, d, kw):
    c = Paged(lens, heads, d, 60 + d)
    total = sum(new)
    qb = _query_bits(total, heads * group, d, 61)
    q = bf16(qb)
    m = max(lens) + 3
    m = min(m, c.table.shape[1] * PAGE)
    _, lse = nv.kv_attention(q, c.cache, c.table_t, c.lens_t, starts(new), max(new), m, **kw)
    prior = torch.rand(len(lens), heads, m, device=DEV)
    got = nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, starts(new), max(new), m, prior=prior, **kw)
    bare = nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, starts(new), max(new), m, **kw)
    again = nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, starts(new), max(new), m, prior=prior, **kw)
    place = prior.clone()
    nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, starts(new), max(new), m, prior=place, out=place, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got, again) and torch.equal(got, place)
    got, bare, prior = (x.cpu().numpy().astype(np.float64) for x in (got, bare, prior))
    l64 = lse.cpu().numpy().astype(np.float64)
    q64 = bf16_bits_to_f64(qb)
    at = 0
    for s, n in enumerate(lens):
        assert not got[s, :, n:].any() and not bare[s, :, n:].any()
        for h in range(heads):
            want, size = np.zeros(n), np.zeros(n)
            for g in range(group):
                w, z = okv.slot_weights(q64[at:at + new[s], h * group + g], c.k[s][h], l64[at:at + new[s], h * group + g],
                                        d ** -0.5, **kw)
                want, size = want + w, size + z
            # each term's relative error as for the scores (lse is an input; z - lse rounds once more,
            # at |z| <= size), and one rounding a term and for the prior
            cap = kw.get("softcap", 0.0)
            tol = 2 * (d + 8) * 2.0 ** -24 * size + (2.0 ** -20 + 8 * cap * 2.0 ** -23 + (new[s] * group + 2) * 2.0 ** -24) * want
            tol = tol + np.abs(l64[at:at + new[s]][np.isfinite(l64[at:at + new[s]])]).max(initial=0.0) * 2.0 ** -22 * want
            assert np.all(np.abs(bare[s, h, :n] - want) <= tol + 1e-30), (s, h)
            total_w = prior[s, h, :n] + want
            assert np.all(np.abs(got[s, h, :n] - total_w) <= tol + 2.0 ** -23 * total_w + 1e-30), (s, h)
        at += new[s]


def _weights(g, shape):
    w = g.random(shape, dtype=np.float32)
    w[w < 0.3] = 0.0                                           # ties at zero
    w[(w > 0.5) & (w < 0.6)] = np.float32(0.55)                # and elsewhere
    return w


@pytest.mark.parametrize("lens,heads,d,keep,sink,recent", [
    ([10], 1, 64, 4, 0, 0), ([200, 33, 64], 2, 128, 64, 4, 16), ([130, 65, 1], 1, 256, 65, 0, 64),
    ([3000, 1025, 2049, 1024], 1, 64, 1000, 1, 500), ([100], 2, 64, 100, 3, 3), ([0, 7], 1, 64, 5, 5, 0),
    ([500], 1, 64, 70, 35, 35), ([90, 200], 1, 64, 1, 0, 0),
])
def test_evict(lens, heads, d, keep, sink, recent):
    g = workload.rng(70)
    need = -(-keep // PAGE)
    c = Paged(lens, heads, d, 71, extra=need * len(lens))
    w = _weights(g, (len(lens), heads, max(max(lens), 1)))
    w[0, 0, ::7] = np.nan
    w[0, 0, 1::11] = -0.0
    w[-1, -1, ::5] = np.inf
    w[-1, -1, 1::5] = -np.inf
    dst_table = np.array(c.free, np.int32).reshape(len(lens), need)
    before = c.data.cpu().numpy().copy()
    kept, kept_w, new_lens = nv.kv_evict(torch.from_numpy(w).to(DEV), c.cache, c.table_t, c.lens_t, int32(dst_table), keep,
                                         sink=sink, recent=recent)
    torch.cuda.synchronize()
    kept, kept_w, after = kept.cpu().numpy(), kept_w.cpu().numpy(), c.data.cpu().numpy()
    assert new_lens.cpu().tolist() == [min(n, keep) for n in lens]
    for s, n in enumerate(lens):
        for h in range(heads):
            want = okv.evict(w[s, h], n, keep, sink, recent)
            m = len(want)
            assert np.array_equal(kept[s, h, :m], want), (s, h)
            assert np.all(kept[s, h, m:] == -1) and not kept_w[s, h, m:].any()
            assert np.array_equal(kept_w[s, h, :m], w[s, h, want], equal_nan=True)
            if m == 0:
                continue
            full = -(-m // PAGE) * PAGE
            src = stored(before, c.table[s], n, h, d)
            got = stored(after, dst_table[s], full, h, d)
            for a, b in zip(src, got):
                assert np.array_equal(a[want], b[:m]), (s, h)
                assert not b[m:].any()
            for a, b in zip(src, stored(after, c.table[s], n, h, d)):
                assert np.array_equal(a, b)                    # the sources are as they were


def test_evict_into_another_cache_then_attend():
    # what attention sees of the smaller cache is what the oracle computes of the kept rows
    lens, keep = [700, 90], 128
    c = Paged(lens, 2, 64, 80)
    qb = _query_bits(2, 4, 64, 81)
    q = bf16(qb)
    _, lse = nv.kv_attention(q, c.cache, c.table_t, c.lens_t, starts([1, 1]), 1, 700)
    w = nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, starts([1, 1]), 1, 700)
    small = nv.KvCache.empty(4, 2, 64, c.k_scale, c.v_scale)
    dst = int32([[3, 1], [0, 2]])
    kept, _, new_lens = nv.kv_evict(w, c.cache, c.table_t, c.lens_t, dst, keep, sink=2, recent=30, dst=small)
    rows = kept.cpu().numpy()
    for s in range(2):
        m = min(lens[s], keep)
        c.k[s] = np.stack([c.k[s][h][rows[s, h, :m]] for h in range(2)])
        c.v[s] = np.stack([c.v[s][h][rows[s, h, :m]] for h in range(2)])
    c.lens, c.cache, c.table_t, c.lens_t = [128, 90], small, dst, new_lens
    out, lse = _attend(c, qb, [1, 1])
    _check(c, qb, [1, 1], out, lse)


def test_evict_of_more_slots_than_registers_hold():
    # 65536 slots' keys fit the selection's registers; longer sequences are read again for each step
    g = workload.rng(72)
    n, keep = 70000, 100
    cache = nv.KvCache.empty(-(-n // PAGE) + 2, 1, 64, 1.0, 1.0)
    table = int32(np.arange(-(-n // PAGE))[None])
    w = _weights(g, (1, 1, n))
    kept, kept_w, new_lens = nv.kv_evict(torch.from_numpy(w).to(DEV), cache, table, int32([n]), int32([[1094, 1095]]), keep,
                                         sink=3, recent=10)
    want = okv.evict(w[0, 0], n, keep, 3, 10)
    assert np.array_equal(kept.cpu().numpy()[0, 0], want) and new_lens.tolist() == [keep]
    assert np.array_equal(kept_w.cpu().numpy()[0, 0], w[0, 0, want])


@pytest.mark.parametrize("n", [4097, 9001, 16384, 16385, 40000, 65535, 65537])
@pytest.mark.parametrize("kind", ["ties", "zeros", "one value", "signs"])
def test_evict_selection_at_every_length(n, kind):
    """Which slots stay of long sequences, whose keys are held or read again, with many equal weights."""
    g = workload.rng(73)
    need = -(-n // PAGE)
    lens = [n, n - 4000, 700]
    w = {"ties": lambda: _weights(g, (3, 1, n)), "zeros": lambda: np.zeros((3, 1, n), np.float32),
         "one value": lambda: np.full((3, 1, n), 0.125, np.float32),
         "signs": lambda: g.standard_normal((3, 1, n)).astype(np.float32)}[kind]()
    w[:, :, 5::97] = np.nan
    w[:, :, 6::89] = -np.inf
    keep = 1300
    pages = -(-keep // PAGE)
    cache = nv.KvCache.empty(need + 3 * pages, 1, 64, 1.0, 1.0)
    table = int32(np.tile(np.arange(need), (3, 1)))           # the sequences read the same pages
    dst = int32(need + np.arange(3 * pages).reshape(3, pages))
    kept, kept_w, new_lens = nv.kv_evict(torch.from_numpy(w).to(DEV), cache, table, int32(lens), dst, keep, sink=7, recent=64)
    kept, kept_w = kept.cpu().numpy(), kept_w.cpu().numpy()
    assert new_lens.tolist() == [min(x, keep) for x in lens]
    for i, x in enumerate(lens):
        want = okv.evict(w[i, 0], x, keep, 7, 64)
        assert np.array_equal(kept[i, 0, :len(want)], want), i
        assert np.array_equal(kept_w[i, 0, :len(want)], w[i, 0, want], equal_nan=True)


def test_slot_weights_do_not_depend_on_the_launch():
    # a large bound on the lengths gives a wavefront two pages, a small one one; rows of more blocks are added in order
    lens = [300, 0, 64, 65, 129, 257] * 6
    c = Paged(lens, 8, 64, 64)
    wide = int32(np.pad(c.table_t.cpu().numpy(), ((0, 0), (0, 40))))
    for new in (1, 7):
        news = [min(new, n) for n in lens]
        q = bf16(_query_bits(sum(news), 16, 64, 65))
        args = (c.cache, wide, c.lens_t, starts(news), new)
        _, lse = nv.kv_attention(q, *args, 320)
        small = nv.kv_weights(q, lse, *args, 320)
        large = nv.kv_weights(q, lse, *args, 2500)
        torch.cuda.synchronize()
        assert torch.equal(small, large[:, :, :320]) and not large[:, :, 320:].any()


@pytest.mark.parametrize("d,new,kw", [(64, 40, {}), (128, 70, dict(window=90)), (256, 40, dict(softcap=9.0)), (128, 64, dict(causal=False))])
def test_slot_weights_of_many_rows_in_every_launch(d, new, kw):
    # few pages: a workgroup's wavefronts share one; more: a page each; many and one block of rows: four each
    lens = [300, 64, 129, 257, 65, 0] * 6
    c = Paged(lens, 8, d, 66)
    wide = int32(np.pad(c.table_t.cpu().numpy(), ((0, 0), (0, 20))))
    news = [min(new, n) for n in lens]
    q = bf16(_query_bits(sum(news), 16, d, 67))
    args = (c.cache, wide, c.lens_t, starts(news), new)
    _, lse = nv.kv_attention(q, *args, 320, **kw)
    one = nv.kv_weights(q, lse, *args, 320, **kw)
    four = nv.kv_weights(q, lse, *args, 1600, **kw)
    part = sum(news[:3])
    shared = nv.kv_weights(q[:part], lse[:part], c.cache, wide[:3].contiguous(), c.lens_t[:3], starts(news[:3]), new, 320, **kw)
    torch.cuda.synchronize()
    assert torch.equal(one, four[:, :, :320]) and not four[:, :, 320:].any()
    # sums of at most 140 numbers that are not negative, in two orders: 2 * 140 * 2^-24 of the sum
    assert torch.allclose(shared, one[:3], rtol=2e-5, atol=0)


def test_sequences_beyond_the_host_s_bounds_are_held_to_them():
    # nothing is read or written past what the launch was sized for
    c = Paged([300, 40], 1, 64, 91)
    q = bf16(_query_bits(41, 2, 64, 92))
    out, lse = nv.kv_attention(q, c.cache, c.table_t, c.lens_t, starts([40, 1]), 8, 128)
    w = nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, starts([40, 1]), 8, 128)
    torch.cuda.synchronize()
    assert w.shape == (2, 1, 128)


def test_no_sequences_and_no_tokens():
    c = nv.KvCache.empty(1, 1, 64, 1.0, 1.0)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    empty = torch.empty((0, 1), dtype=torch.int32, device=DEV)
    no = torch.empty((0,), dtype=torch.int32, device=DEV)
    out, lse = nv.kv_attention(none, c, empty, no, int32([0]), 0, 0)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    nv.kv_append(c, none[:, :1], none[:, 1:], empty, no, int32([0]))
    k, v = nv.kv_read(c, empty, no, int32([0]), 0)
    assert k.shape == (0, 1, 64)
    out, lse = nv.kv_attention(none, c, int32([[0]]), int32([0]), int32([0, 0]), 0, 0)
    torch.cuda.synchronize()
    assert not c.data.any()

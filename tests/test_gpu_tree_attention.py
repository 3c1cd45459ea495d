"""Attention of the nodes of drafted trees over the paged NVFP4 cache (gpu),
against the float64 oracle.

Tolerances are those of test_gpu_kv.py, which derives them: the arithmetic is the
same, only what a row sees differs."""
import numpy as np
import pytest
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle import bf16_bits_to_f64
from oracle import draft as odraft
from tests._kv import DEV, Paged, bf16, int32, starts
from tests.test_gpu_draft import _parents
from tests.test_gpu_kv import _eps, _query_bits
from tests.test_gpu_kv_ranges import Guarded

pytestmark = pytest.mark.gpu


def _masks(ints, words):
    """Python integers of bits as an int64 tensor [rows, words]."""
    a = np.array([[(m >> 64 * w) & (2 ** 64 - 1) for w in range(words)] for m in ints], np.uint64).reshape(len(ints), words)
    return torch.from_numpy(a.view(np.int64)).to(DEV)


def _of_trees(g, lens, new, near=6):
    """(masks as Python integers, positions) of random trees."""
    masks, positions = [], []
    for n, nq in zip(lens, new):
        for way in odraft.ways(_parents(g, nq, near)):
            masks.append(sum(1 << a for a in way))
            positions.append(n - nq + len(way) - 1)
    return masks, positions


def _wide(c):
    """The cache's tables with rows so long that, by its bounds, a call is one for the tiles of many rows; what is added is no page."""
    pitch = 1 << 14
    table = torch.full((len(c.lens), pitch), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table_t.shape[1]] = c.table_t
    return table, pitch * 64


def _attend(c, qbits, new, masks, positions, words=None, strided=False, max_q=None, max_kv=None, wide=False, **kw):
    q = bf16(qbits)
    if strided:                                              # a view of a fused projection's output
        total, heads, d = q.shape
        fused = torch.full((total, heads * d + 2 * c.heads * d), float("nan"), dtype=torch.bfloat16, device=DEV)
        fused[:, :heads * d] = q.reshape(total, heads * d)
        q = fused[:, :heads * d].view(total, heads, d)
    max_q = max_q or max(max(new), 1)
    words = words or -(-max_q // 64)
    table = c.table_t
    if wide:
        table, max_kv = _wide(c)
    out, lse = nv.kv_tree_attention(q, c.cache, table, c.lens_t, starts(new), _masks(masks, words),
                                    None if positions is None else int32(positions), max_q,
                                    max_kv if max_kv is not None else max(max(c.lens), 1), **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def _check(c, qbits, new, masks, positions, out, lse, window=0, softcap=0.0, scale=None):
    q = bf16_bits_to_f64(qbits)
    heads, d = q.shape[1], c.d
    scale = d ** -0.5 if scale is None else scale
    at = 0
    for s, n in enumerate(c.lens):
        rows = slice(at, at + new[s])
        seen = odraft.visible(n, masks[rows], positions[rows] if positions is not None else None, window)
        for h in range(heads):
            k, v = c.k[s][h // (heads // c.heads)], c.v[s][h // (heads // c.heads)]
            o, l, spread, size = odraft.attention(q[rows, h], k, v, seen, scale, softcap)
            eps = _eps(size, d, softcap)[:, None]
            top = np.abs(v).max() if n else 0.0
            tol = 2.0 ** -8 * np.abs(o) + (eps + 2.0 ** -10) * spread + (n + 1) * 2.0 ** -24 * top
            err = np.abs(out[rows, h] - o)
            assert np.all(err <= tol), (s, h, float((err / np.maximum(tol, 1e-300)).max()))
            empty = ~np.isfinite(l)
            got = lse[rows, h]
            assert np.array_equal(np.isneginf(got), empty), (s, h)
            assert np.all(out[rows, h][empty] == 0.0)
            lim = eps[:, 0] + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(empty, 0, l)))
            assert np.all(np.abs(got - l)[~empty] <= lim[~empty]), (s, h)
        at += new[s]


CASES = [
    # lens, new, kv heads, group, D, options: up to 16, 32, 64 and more rows a kv head
    ([1], [1], 1, 1, 64, {}),
    ([1, 2, 63, 64, 65], [1, 2, 3, 4, 4], 2, 4, 128, {}),
    ([700, 5, 129], [16, 5, 7], 2, 1, 64, {}),
    ([300, 31, 16], [16, 8, 16], 1, 2, 256, {}),
    ([300, 131], [12, 9], 2, 4, 128, {}),
    ([300, 64, 200], [16, 13, 1], 1, 4, 256, {}),
    ([300, 131, 64], [64, 40, 64], 2, 4, 128, {}),
    ([500, 256, 300], [256, 255, 129], 1, 2, 64, {}),
    ([400, 90], [200, 65], 1, 1, 256, {}),
    ([300, 70], [70, 33], 1, 8, 64, {}),
    ([333, 64, 65, 1], [9, 2, 30, 1], 2, 2, 128, dict(window=1)),
    ([333, 64, 65], [20, 2, 60], 1, 4, 128, dict(window=67)),
    ([333, 70], [30, 64], 1, 3, 64, dict(window=5)),
    ([333, 70], [100, 30], 2, 1, 256, dict(window=100, softcap=5.0)),
    ([150, 260], [64, 3], 1, 8, 128, dict(softcap=30.0)),
    ([0, 5, 0], [1, 1, 0], 1, 2, 64, {}),                      # nothing cached: empty rows
    ([3, 2], [8, 5], 1, 2, 64, {}),                            # more nodes than slots
    ([40, 20], [100, 70], 1, 1, 128, dict(window=9)),
    ([500, 40], [0, 3], 2, 2, 128, {}),                        # a sequence without nodes
    ([64, 128], [64, 64], 1, 1, 64, {}),                       # nothing, or a whole page, before the tree
    ([5000, 40, 2100], [16, 3, 9], 1, 4, 128, {}),             # parts of pages
    ([9000, 70], [60, 64], 1, 4, 64, {}),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,new,heads,group,d,kw", CASES)
def test_tree_attention(lens, new, heads, group, d, kw, wide):
    g = workload.rng(sum(lens) + d)
    c = Paged(lens, heads, d, 400 + sum(lens))
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(sum(new), heads * group, d, 27 + d)
    out, lse = _attend(c, qb, new, masks, positions, strided=len(lens) % 2 == 0, wide=wide, **kw)
    _check(c, qb, new, masks, positions, out, lse, **kw)
    again = _attend(c, qb, new, masks, positions, wide=wide, **kw)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("new,group,d", [([12, 40], 2, 128), ([64, 33], 1, 64), ([130, 256], 1, 64), ([20, 9], 2, 256)])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("wide", [False, True])
def test_masks_that_are_no_trees(new, group, d, window, wide):
    # any bits: none at all, later nodes, bits beyond the last node, positions outside the tree
    lens = [300, 256]
    g = workload.rng(sum(new) + d)
    c = Paged(lens, 1, d, 500 + d)
    rows = sum(new)
    masks = [int.from_bytes(g.bytes(32), "little") & int.from_bytes(g.bytes(32), "little") for _ in range(rows)]
    for i in range(0, rows, 5):
        masks[i] = 0
    positions = g.integers(-100, 500, rows).tolist()
    positions[1], positions[2] = 2 ** 31 - 1, -(2 ** 31)
    qb = _query_bits(rows, group, d, 5)
    out, lse = _attend(c, qb, new, masks, positions, words=4, window=window, wide=wide and window == 0)
    _check(c, qb, new, masks, positions, out, lse, window=window)


@pytest.mark.parametrize("wide", [False, True])
def test_a_row_that_sees_nothing(wide):
    # nothing before the tree, and no bits
    for new in ([4], [20], [100]):
        c = Paged(new, 1, 64, 12)
        masks = [0 if i % 3 else 1 << i for i in range(new[0])]
        qb = _query_bits(new[0], 2, 64, 13)
        out, lse = _attend(c, qb, new, masks, None, wide=wide)
        _check(c, qb, new, masks, None, out, lse)
        assert np.isneginf(lse[1]).all() and not out[1].any()


@pytest.mark.parametrize("wide", [False, True])
def test_a_chain_sees_what_causal_attention_sees(wide):
    for new in ([1, 3], [9, 16], [100, 30]):
        lens = [700, 130]
        c = Paged(lens, 2, 128, 14)
        masks = [(2 << i) - 1 for n in new for i in range(n)]
        positions = [n - nq + i for n, nq in zip(lens, new) for i in range(nq)]
        qb = _query_bits(sum(new), 8, 128, 15)
        out, lse = _attend(c, qb, new, masks, positions, wide=wide)
        _check(c, qb, new, masks, positions, out, lse)
        from tests.test_gpu_kv import _check as check_causal
        check_causal(c, qb, new, out, lse)


def test_bounds_that_exceed_the_trees():
    lens, new = [100, 90], [3, 20]
    g = workload.rng(6)
    c = Paged(lens, 2, 128, 5)
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(23, 4, 128, 6)
    for max_q in (20, 50, 256):
        out, lse = _attend(c, qb, new, masks, positions, max_q=max_q, max_kv=c.table.shape[1] * 64)
        _check(c, qb, new, masks, positions, out, lse)


@pytest.mark.parametrize("wide", [False, True])
def test_trees_beyond_the_bound_are_taken_for_their_first_nodes(wide):
    lens, new, most = [200, 90], [30, 10], 12
    g = workload.rng(7)
    c = Paged(lens, 1, 64, 8)
    masks, positions = _of_trees(g, lens, [most, 10])
    at = [i for i in range(most)] + [30 + i for i in range(10)]
    all_masks, all_positions = [0] * 40, [0] * 40
    for i, m, p in zip(at, masks, positions):
        all_masks[i], all_positions[i] = m, p
    qb = _query_bits(40, 4, 64, 9)
    out = Guarded((40, 4, 64), torch.bfloat16)
    untouched = out.t.clone()
    lse = torch.full((40, 4), 7.0, device=DEV)
    table, max_kv = _wide(c) if wide else (c.table_t, 200)
    nv.kv_tree_attention(bf16(qb), c.cache, table, c.lens_t, starts(new), _masks(all_masks, 1), int32(all_positions), most, max_kv,
                         out=out.t, lse=lse)
    torch.cuda.synchronize()
    got = out.check().float().cpu().numpy().astype(np.float64)[at]
    _check(c, qb[at], [most, 10], masks, positions, got, lse.cpu().numpy().astype(np.float64)[at])
    assert torch.equal(out.t[most:30].view(torch.int16), untouched[most:30].view(torch.int16)) and bool((lse[most:30] == 7.0).all())


@pytest.mark.parametrize("wide", [False, True])
def test_nan_and_infinite_queries_stay_in_their_rows(wide):
    for new in ([5], [20], [40], [120]):
        c = Paged([250], 1, 64, 8)
        g = workload.rng(9)
        masks, positions = _of_trees(g, [250], new)
        qb = _query_bits(new[0], 3, 64, 9)
        clean = _attend(c, qb, new, masks, positions, wide=wide)
        bad = qb.copy()
        bad[1, 1, 3], bad[3, 2, 0] = 0x7FC0, 0x7F80
        out, lse = _attend(c, bad, new, masks, positions, wide=wide)
        hit = np.zeros((new[0], 3), bool)
        hit[1, 1] = hit[3, 2] = True
        assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
        assert np.array_equal(out[~hit], clean[0][~hit]) and np.array_equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new", [[9, 8], [30, 16], [90, 64]])
def test_pages_outside_the_cache(new, wide):
    # a page number that the cache does not have stands for slots that nothing sees, in and before the tree
    lens = [330, 200]
    c = Paged(lens, 1, 64, 12)
    g = workload.rng(13)
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(sum(new), 2, 64, 3)
    table = c.table.copy()
    table[0, 1], table[1, 2] = 10 ** 6, -7
    c.table_t = int32(table)
    out, lse = _attend(c, qb, new, masks, positions, wide=wide)
    q, at = bf16_bits_to_f64(qb), 0
    for s, n in enumerate(lens):
        rows = slice(at, at + new[s])
        seen = odraft.visible(n, masks[rows], positions[rows], 0)
        seen[:, 64:128 if s == 0 else 64] = False
        if s == 1:
            seen[:, 128:192] = False
        for h in range(2):
            o, l, spread, size = odraft.attention(q[rows, h], c.k[s][0], c.v[s][0], seen, 0.125)
            tol = 2.0 ** -8 * np.abs(o) + (_eps(size, 64, 0.0)[:, None] + 2.0 ** -10) * spread + (n + 1) * 2.0 ** -24 * np.abs(c.v[s][0]).max()
            assert np.all(np.abs(out[rows, h] - o) <= tol)
        at += new[s]


@pytest.mark.parametrize("wide", [False, True])
def test_negative_and_zero_scales(wide):
    for new in ([5, 4], [40, 30], [128, 20]):
        lens = [300, 170]
        c = Paged(lens, 1, 128, 23)
        masks, positions = _of_trees(workload.rng(3), lens, new)
        qb = _query_bits(sum(new), 2, 128, 24)
        for scale in (-0.2, 0.0):
            out, lse = _attend(c, qb, new, masks, positions, scale=scale, wide=wide)
            _check(c, qb, new, masks, positions, out, lse, scale=scale)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new", [[8, 9], [16, 12], [64, 50]])
def test_on_another_stream_and_in_a_graph(new, wide):
    lens = [3000, 100]
    c = Paged(lens, 2, 128, 21)
    masks, positions = _of_trees(workload.rng(22), lens, new)
    qb = _query_bits(sum(new), 8, 128, 22)
    want, want_lse = _attend(c, qb, new, masks, positions, wide=wide)
    table, most = _wide(c) if wide else (c.table_t, 3000)
    q, st, total = bf16(qb), starts(new), sum(new)
    m, p = _masks(masks, 1), int32(positions)
    out = torch.empty((total, 8, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((total, 8), dtype=torch.float32, device=DEV)
    ws = torch.empty(nv.kv_tree_attention_workspace(c.cache, q, table, c.lens_t, st, max(new), most), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nv.kv_tree_attention(q, c.cache, table, c.lens_t, st, m, p, max(new), most, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert np.array_equal(out.float().cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv_tree_attention(q, c.cache, table, c.lens_t, st, m, p, max(new), most, out=out, lse=lse, workspace=ws)
    for _ in range(4):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy(), want) and np.array_equal(lse.cpu().numpy(), want_lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new", [[5, 9], [40, 30], [16, 14]])
def test_descending_starts_touch_nothing_beyond_the_arrays(new, wide):
    d, heads, total = 64, 4, sum(new) + 20
    c = Paged([3000, 90, 500], 2, d, 221)
    g = workload.rng(31)
    masks = _masks([int.from_bytes(g.bytes(8), "little") for _ in range(total)], 1)
    q = bf16(_query_bits(total, heads, d, 223))
    table, most = _wide(c) if wide else (c.table_t, 3000)
    for order in ([total, 0, new[0], new[0] + new[1]], [7, 3, total, 0], [new[0] + 1, new[0] + 2, 0, new[0]]):
        st = int32(order)
        out, lse = Guarded((total, heads, d), torch.bfloat16), Guarded((total, heads), torch.float32)
        n = nv.kv_tree_attention_workspace(c.cache, q, table, c.lens_t, st, max(new), most)
        ws = Guarded((n,), torch.uint8) if n else None
        nv.kv_tree_attention(q, c.cache, table, c.lens_t, st, masks, None, max(new), most, out=out.t, lse=lse.t, workspace=ws and ws.t)
        torch.cuda.synchronize()
        for x in (out, lse, *([ws] if ws else [])):
            x.check()


@pytest.mark.parametrize("most,group,wide", [(5, 2, False), (5, 8, True), (12, 8, True)])
def test_many_sequences_of_very_different_lengths(most, group, wide):
    # pages planned from the lengths, and more sequences than a wavefront has lanes
    g = workload.rng(31)
    lens = [int(x) for x in np.exp(g.uniform(0, np.log(2500), 70))]
    lens[3], lens[40], lens[-1] = 0, 12000, 1
    new = [min(int(g.integers(1, most)), n) for n in lens]
    new[-2] = min(most, lens[-2])
    c = Paged(lens, 4, 64, 32)
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(sum(new), 4 * group, 64, 33)
    out, lse = _attend(c, qb, new, masks, positions, wide=wide)
    _check(c, qb, new, masks, positions, out, lse)
    again = _attend(c, qb, new, masks, positions, wide=wide)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])


def test_many_short_sequences():
    # none has more pages than a workgroup takes whole, and there are enough of them for the tiles
    g = workload.rng(41)
    lens = [int(g.integers(1, 250)) for _ in range(600)]
    new = [min(n, int(g.integers(1, 12))) for n in lens]
    c = Paged(lens, 8, 64, 42)
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(sum(new), 64, 64, 43)
    out, lse = _attend(c, qb, new, masks, positions, max_q=256)
    some = [0, 1, 299, 300, 598, 599]
    at = np.concatenate([[0], np.cumsum(new)])
    rows = np.concatenate([np.arange(at[s], at[s + 1]) for s in some])
    few = type("Few", (), dict(lens=[lens[s] for s in some], d=64, heads=8, k=[c.k[s] for s in some], v=[c.v[s] for s in some]))
    _check(few, qb[rows], [new[s] for s in some], [masks[r] for r in rows], [positions[r] for r in rows], out[rows], lse[rows])
    assert np.isfinite(out).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("d,window,softcap", [(64, 100, 0.0), (64, 1, 0.0), (128, 70, 6.0), (256, 130, 0.0)])
def test_windows_in_tiles_of_many_rows(d, window, softcap):
    g = workload.rng(51)
    lens = [int(g.integers(1, 400)) for _ in range(40)]
    new = [min(n, int(g.integers(1, 40))) for n in lens]
    c = Paged(lens, 8, d, 52)
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(sum(new), 64, d, 53)
    # a bound of 256 nodes makes it a call for the tiles
    out, lse = _attend(c, qb, new, masks, positions, max_q=256, window=window, softcap=softcap)
    some = [0, 7, 20, 39]
    at = np.concatenate([[0], np.cumsum(new)])
    rows = np.concatenate([np.arange(at[s], at[s + 1]) for s in some])
    few = type("Few", (), dict(lens=[lens[s] for s in some], d=d, heads=8, k=[c.k[s] for s in some], v=[c.v[s] for s in some]))
    _check(few, qb[rows], [new[s] for s in some], [masks[r] for r in rows], [positions[r] for r in rows], out[rows], lse[rows], window=window,
           softcap=softcap)
    assert np.isfinite(out).all() and np.isfinite(lse).all()


def test_more_rows_than_32_bits_of_threads():
    # 4096 trees over the same short cache, then one over a long one, whose rows are those from 2^25 on (a wavefront each
    # would be more threads than a launch has)
    lens, nodes, heads, many = [130, 8000], 128, 64, 4096
    c = Paged(lens, 1, 64, 41, v_scale=0.5)
    masks, _ = _of_trees(workload.rng(42), lens, [nodes, nodes])
    total = (many + 1) * nodes
    qb = _query_bits(2 * nodes, heads, 64, 43)
    q = torch.empty((total, heads, 64), dtype=torch.bfloat16, device=DEV)
    ends = bf16(qb)
    q[:many * nodes].view(many, nodes, heads, 64)[:] = ends[:nodes]
    q[many * nodes:] = ends[nodes:]
    m = _masks(masks, 2)
    m = torch.cat([m[:nodes].repeat(many, 1), m[nodes:]])
    table = torch.cat([c.table_t[:1].repeat(many, 1), c.table_t[1:]])
    out, lse = nv.kv_tree_attention(q, c.cache, table, int32([lens[0]] * many + [lens[1]]), starts([nodes] * (many + 1)), m, None, nodes,
                                    lens[1])
    pick = torch.cat([torch.arange(nodes), torch.arange(total - nodes, total)]).to(DEV)
    _check(c, qb, [nodes, nodes], masks, None, out[pick].float().cpu().numpy().astype(np.float64), lse[pick].cpu().numpy().astype(np.float64))
    # the trees are alike, and the parts that some were joined of change a sum's last bits alone
    first = out[:nodes].float()
    for s in (1, 7, 2047, 4095):
        assert float((out[s * nodes:(s + 1) * nodes].float() - first).abs().max()) <= 2.0 ** -6 * float(first.abs().max())

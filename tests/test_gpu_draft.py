"""The whole numbers and the moves of a verify round on the GPU (gpu): page
tables, trees, accepted branches and moved slots, equal to the oracle's, with
guards around what a call may write."""
import numpy as np
import pytest
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle import draft as odraft
from tests._kv import DEV, PAGE, Paged, int32, starts, stored
from tests.test_gpu_kv_ranges import Guarded

pytestmark = pytest.mark.gpu


# ---- page tables

def _pool(g, seqs, pitch, most_held, spare):
    """A pool in which the sequences hold up to most_held pages each: (pool, state, table, held)."""
    held = g.integers(0, min(most_held, pitch) + 1, seqs)
    pages = int(held.sum()) + spare
    order = g.permutation(pages).tolist()
    table = np.full((seqs, pitch), -1, np.int32)
    for s, n in enumerate(held):
        table[s, :n] = [order.pop() for _ in range(n)]
    cap = pages + 3
    head = int(g.integers(0, cap))
    pool = np.full(cap, -7, np.int32)
    pool[(head + np.arange(len(order))) % cap] = order
    return pool, np.array([head, len(order)], np.int32), table, held.astype(np.int32)


def _step(pool, state, table, held, keep, fresh, total, guard=True):
    """One call: (the oracle's results, the library's as lists)."""
    want = odraft.pages(pool, state, table, held, keep, fresh, total)
    seqs = len(held)
    ins = [Guarded(np.shape(a), torch.int32, int32(a)) for a in (pool, table)]
    outs = [Guarded((n,), torch.int32) for n in (2, seqs, seqs, seqs + 1, total, total)]
    step = nv.kv_pages(ins[0].t, int32(state), ins[1].t, int32(held), int32(keep), int32(fresh), total,
                       out=nv.KvStep(*(o.t for o in outs)))
    torch.cuda.synchronize()
    p, t = (i.check().cpu().numpy() for i in ins)
    st, hd, lens, qs, slots, pos = (o.check().cpu().numpy().tolist() for o in outs)
    assert step.slots.data_ptr() == outs[4].t.data_ptr()
    return want, (p.tolist(), st, t, hd, lens, qs, slots, pos)


def _same(want, got):
    names = ("pool", "state", "table", "held", "kv_lens", "q_starts", "slots", "positions")
    for name, a, b in zip(names, want, got):
        assert np.array_equal(np.asarray(a), np.asarray(b)), (name, a, b)


@pytest.mark.parametrize("seqs,pitch,held,fresh,spare,total", [
    (1, 1, 0, 1, 1, 1),
    (1, 4, 2, 100, 9, 100),
    (48, 9, 8, 1, 60, 48),
    (64, 9, 8, 70, 100, 64 * 70),          # more tokens than one workgroup fills
    (64, 9, 8, 70, 20, 64 * 70),           # too few pages: some are not granted
    (64, 9, 8, 70, 400, 900),              # too few rows
    (70, 3, 3, 150, 400, 70 * 150),        # some do not fit a table row
    (1024, 5, 4, 3, 900, 4096),
    (1025, 5, 4, 3, 700, 4097),            # a second block of sequences
    (2600, 4, 3, 90, 900, 60000),
    (5, 300, 290, 8191, 900, 40000),
    (7, 6, 5, 0, 0, 0),
])
def test_pages(seqs, pitch, held, fresh, spare, total):
    g = workload.rng(seqs * 7 + total)
    pool, state, table, held = _pool(g, seqs, pitch, held, spare)
    keep = (g.random(seqs) * (64 * held + 1)).astype(np.int32)
    keep[g.random(seqs) < 0.2] = 0
    new = g.integers(0, fresh + 1, seqs).astype(np.int32)
    _same(*_step(pool, state, table, held, keep, new, total))


def test_pages_take_inputs_into_their_ranges():
    big = 2 ** 31 - 1
    pool, table = np.arange(20, 32, dtype=np.int32), np.arange(12, dtype=np.int32).reshape(4, 3)
    for state in ([-5, 100], [big, 4], [12, -1], [-(2 ** 31), big], [3, 12]):
        for held, keep, fresh in (([9, -2, 1, 3], [big, 5, -7, 100], [0, 1, -4, 90]), ([0, 0, 0, 0], [0, 9, big, 0], [big, big, 64, 65]),
                                  ([3, 3, 3, 3], [0, 0, 1, 192], [0, 0, 0, 0])):
            _same(*_step(pool, state, table, held, keep, fresh, 100))
    # page numbers that have no place in a slot's number
    bad = np.array([[-1, 1 << 25, (1 << 25) - 1]], np.int32)
    want, got = _step(pool, [0, 0], bad, [3], [0], [192], 200)
    _same(want, got)
    assert got[6][0] == got[6][64] == -1 and got[6][128] == ((1 << 25) - 1) * 64


def test_pages_of_no_sequence_and_without_maps():
    step = nv.kv_pages(int32([1, 2]), int32([1, 1]), torch.zeros(0, 3, dtype=torch.int32, device=DEV), int32([]), int32([]), int32([]), 5)
    assert step.state.tolist() == [1, 1] and step.q_starts.tolist() == [0] and step.slots.tolist() == step.positions.tolist() == [-1] * 5
    from verify_nvfp4_w4a16_amd import drafting
    table, outs = int32([[3, -1]]), [int32([9] * n) for n in (2, 1, 1, 2)]
    a = [int32(x) for x in ([5, 6], [0, 2], [1], [64], [3])]
    p = drafting._Pages(a[0].data_ptr(), a[1].data_ptr(), 2, table.data_ptr(), 2, a[2].data_ptr(), a[3].data_ptr(), a[4].data_ptr(), 1, 8)
    assert drafting._draft().nvfp4_kv_pages(p, *(o.data_ptr() for o in outs), None, None, None) == nv.OK
    torch.cuda.synchronize()
    assert table.tolist() == [[3, 5]] and [o.tolist() for o in outs] == [[1, 1], [2], [67], [0, 3]]


def test_pages_in_a_graph_that_carries_its_state_on():
    """Three captured steps, each on what the last one left, replayed with eager work between."""
    g = workload.rng(5)
    pool, state, table, held = _pool(g, 40, 6, 3, 80)
    tensors = [int32(x) for x in (pool, state, table, held)]
    keep, fresh = int32(np.minimum(64 * held, 100)), int32(g.integers(0, 60, 40))
    out = nv.KvStep(tensors[1], tensors[3], keep, int32([0] * 41), int32([0] * 2400), int32([0] * 2400))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        nv.kv_pages(tensors[0], tensors[1], tensors[2], tensors[3], keep, fresh, 2400, out=out)
    now = [pool, state, table, held, keep.cpu().numpy()]
    for round_ in range(5):
        new = g.integers(0, 60, 40)
        if round_ == 2:
            keep[:20] = 0                                    # half of them end
            now[4] = np.r_[np.zeros(20, np.int32), now[4][20:]]
            new[:20] = 0
        fresh.copy_(int32(new))
        graph.replay()
        torch.cuda.synchronize()
        want = odraft.pages(*now, new, 2400)
        _same(want, (tensors[0].tolist(), out.state.tolist(), tensors[2].cpu().numpy(), out.held.tolist(), out.kv_lens.tolist(),
                     out.q_starts.tolist(), out.slots.tolist(), out.positions.tolist()))
        now = [want[0], want[1], want[2], want[3], np.array(want[4])]
    # nothing was lost on the way
    owned = [int(tensors[2][s, p]) for s in range(40) for p in range(now[3][s])]
    free = [int(now[0][(now[1][0] + i) % len(pool)]) for i in range(now[1][1])]
    assert sorted(owned + free) == list(range(len(pool) - 3))


# ---- trees

def _parents(g, n, near=6):
    return [-1 if i == 0 else int(g.integers(max(0, i - near), i)) for i in range(n)]


def _tree_case(g, new, max_q, wild=0.0):
    parents = []
    for n in new:
        p = _parents(g, n)
        for i in range(n):
            if g.random() < wild:
                p[i] = int(g.choice([-1, -(2 ** 31), i, i + 1, 2 ** 31 - 1, 300]))
        parents += p
    return parents


@pytest.mark.parametrize("new,max_q,wild", [([1], 1, 0.0), ([1, 0, 7], 7, 0.0), ([63, 64, 65], 65, 0.0), ([64, 5], 64, 0.2),
                                            ([256, 1, 129], 256, 0.0), ([200, 255], 255, 0.3), ([90, 40], 50, 0.0), ([9] * 300, 16, 0.1)])
def test_trees(new, max_q, wild):
    g = workload.rng(sum(new) + max_q)
    parents = _tree_case(g, new, max_q, wild)
    if len(new) == 1:
        parents = parents + [5, 5]                           # rows of no sequence
    lens = [int(g.integers(0, 500)) for _ in new]
    total, words = len(parents), -(-max_q // 64)
    masks, positions = Guarded((total, words), torch.int64), Guarded((total,), torch.int32)
    untouched = masks.t.clone(), positions.t.clone()
    nv.kv_tree(int32(parents), int32(lens), starts(new), max_q, masks=masks.t, positions=positions.t)
    torch.cuda.synchronize()
    m, p = masks.check().cpu().numpy().view(np.uint64), positions.check().cpu().numpy()
    at = 0
    for s, n in enumerate(new):
        used = min(n, max_q)
        for i, way in enumerate(odraft.ways(parents[at:at + used])):
            assert m[at + i].tolist() == odraft.mask_words(way, words), (s, i)
            assert p[at + i] == lens[s] - used + len(way) - 1, (s, i)
        # rows beyond max_q stay as they were
        assert torch.equal(masks.t[at + used:at + n], untouched[0][at + used:at + n])
        assert torch.equal(positions.t[at + used:at + n], untouched[1][at + used:at + n])
        at += n
    assert torch.equal(masks.t[at:], untouched[0][at:]) and torch.equal(positions.t[at:], untouched[1][at:])


def test_a_deep_chain_and_a_flat_tree():
    for parents in (list(range(-1, 255)), [-1] + [0] * 255, [-1] * 256):
        masks, positions = nv.kv_tree(int32(parents), int32([300]), int32([0, 256]), 256)
        for i, way in enumerate(odraft.ways(parents)):
            assert masks[i].cpu().numpy().view(np.uint64).tolist() == odraft.mask_words(way, 4)
        assert positions.tolist() == [44 + len(w) - 1 for w in odraft.ways(parents)]


def _accept_case(g, new, vocab):
    drafted = g.integers(-1 if vocab < 5 else 0, vocab, sum(new)).tolist()
    chosen = g.integers(-1 if vocab < 5 else 0, vocab, sum(new)).tolist()
    return drafted, chosen


@pytest.mark.parametrize("new,max_q,vocab", [([1], 1, 9), ([5, 0, 1, 64], 64, 2), ([65, 256, 17], 256, 2), ([30, 200], 200, 4),
                                             ([40, 20], 32, 2), ([12] * 500, 12, 3)])
def test_accept(new, max_q, vocab):
    g = workload.rng(sum(new) * 3 + vocab)
    parents = _tree_case(g, new, max_q, 0.1)
    drafted, chosen = _accept_case(g, new, vocab)
    lens = [int(g.integers(0, 400)) for _ in new]
    seqs = len(new)
    outs = [Guarded(shape, torch.int32) for shape in ((seqs, max_q), (seqs,), (seqs,), (seqs,))]
    nv.tree_accept(int32(drafted), int32(parents), int32(chosen), int32(lens), starts(new), max_q, path=outs[0].t, counts=outs[1].t,
                   token=outs[2].t, new_lens=outs[3].t)
    torch.cuda.synchronize()
    path, counts, token, new_lens = (o.check().cpu().numpy() for o in outs)
    at = longest = 0
    for s, n in enumerate(new):
        used = min(n, max_q)
        i = slice(at, at + used)
        way, last = odraft.accept(drafted[i], parents[i], chosen[i])
        assert path[s].tolist() == way + [-1] * (max_q - len(way)), s
        assert counts[s] == len(way) and token[s] == last and new_lens[s] == max(lens[s] - used + len(way), 0), s
        longest = max(longest, len(way))
        at += n
    assert longest > 1 or max(new) == 1
    # new_lens in kv_lens' place
    where = int32(lens)
    again = nv.tree_accept(int32(drafted), int32(parents), int32(chosen), where, starts(new), max_q, new_lens=where)
    assert torch.equal(again[0], outs[0].t) and where.tolist() == new_lens.tolist()


def test_accept_takes_a_whole_chain():
    n = 256
    tokens = list(range(1, n + 1))
    path, counts, token, new_lens = nv.tree_accept(int32(tokens), int32(range(-1, n - 1)), int32(tokens[1:] + [7]), int32([300]),
                                                   int32([0, n]), n)
    assert path.tolist() == [list(range(n))] and counts.tolist() == [n] and token.tolist() == [7] and new_lens.tolist() == [300]


# ---- moves

def _paths(g, new, max_q, keep=0.4):
    path = np.full((len(new), max_q), -1, np.int32)
    for s, n in enumerate(new):
        used = min(n, max_q)
        nodes = [i for i in range(used) if g.random() < keep]
        path[s, :len(nodes)] = nodes
    return path


def _check_move(c, before, after, new, path, max_q):
    """Every byte of the cache against the oracle: codes and scales of the moved slots, all else as it was."""
    want = before.copy()
    for s, n in enumerate(c.lens):
        nq = min(new[s], max_q)
        for h in range(c.heads):
            old = stored(before, c.table[s], n, h, c.d) if n else None
            for j in range(nq):
                src = int(path[s, j])
                if not 0 <= src < nq:
                    break
                to, at = n - nq + j, n - nq + src
                if to < 0 or at < 0:
                    continue
                pages = [c.table[s, x // PAGE] for x in (to, at)]
                if any(not 0 <= p < len(before) for p in pages):
                    continue
                _put(want[pages[0], h], to % PAGE, [part[at] for part in old], c.d)
    assert np.array_equal(want, after)


def _put(rec, slot, row, d):
    """One slot's (K codes, K scales, V codes, V scales) into a record's bytes."""
    from oracle import kv as okv
    kc, ks, vc, vs = row
    rec[slot * d // 2:(slot + 1) * d // 2] = kc[0::2] | kc[1::2] << 4
    for g in range(d // 16):
        rec[okv.k_scale_index(slot, g, d)], rec[okv.v_scale_index(slot, g, d)] = ks[g], vs[g]
    at = 32 * d + slot // 8 * d * 4 + np.arange(d) * 4 + slot % 8 // 2
    shift = 4 * (slot % 2)
    rec[at] = (rec[at] & (240 >> shift)) | vc << shift


@pytest.mark.parametrize("lens,new,heads,d,keep", [
    ([5], [5], 1, 64, 0.5),
    ([70, 130, 64], [16, 9, 64], 2, 128, 0.4),
    ([200, 333], [100, 200], 1, 256, 0.5),
    ([256, 257, 319, 300], [256, 255, 256, 63], 2, 64, 0.6),
    ([66, 40, 9], [5, 0, 1], 1, 128, 1.0),               # nothing to move
    ([10, 30], [40, 64], 2, 64, 0.7),                    # more nodes than slots: those before slot 0 have none
    ([500, 129], [256, 130], 1, 128, 0.05),
])
def test_move(lens, new, heads, d, keep):
    g = workload.rng(sum(lens) + d)
    c = Paged(lens, heads, d, 70 + sum(new), extra=2)
    before = c.data.cpu().numpy().copy()
    max_q = max(max(new), 1)
    path = _paths(g, new, max_q, keep)
    nv.kv_move(c.cache, c.table_t, c.lens_t, starts(new), int32(path))
    torch.cuda.synchronize()
    _check_move(c, before, c.data.cpu().numpy(), new, path, max_q)


def test_move_of_many_layers_and_bad_pages():
    lens, new, d = [150, 70, 40], [60, 20, 30], 64
    g = workload.rng(9)
    c = Paged(lens, 1, d, 71, extra=1)
    c.table[0, 1], c.table[1, 1] = 10 ** 6, -5
    c.table_t = int32(c.table)
    layers = [Guarded(c.data.shape, torch.uint8, c.data) for _ in range(70)]      # more than one launch takes
    for i, x in enumerate(layers):
        x.t[:, :, 5] = i
    before = [x.t.cpu().numpy().copy() for x in layers]
    path = _paths(g, new, 60, 0.5)
    nv.kv_move([nv.KvCache(x.t, 1, d, 1.0, 1.0) for x in layers], c.table_t, c.lens_t, starts(new), int32(path))
    torch.cuda.synchronize()
    # the oracle reads a sequence's pages one after another: the missing ones as zeros
    for b, x in zip(before, layers):
        shown = np.concatenate([b, np.zeros((1, 1, 72 * d), np.uint8)])
        table = np.where((c.table >= 0) & (c.table < len(b)), c.table, len(b))
        after = np.concatenate([x.check().cpu().numpy(), np.zeros((1, 1, 72 * d), np.uint8)])
        view = type("View", (), dict(lens=lens, heads=1, d=d, table=table))
        _check_view(view, shown, after, new, path, len(b))


def _check_view(c, before, after, new, path, missing):
    want = before.copy()
    for s, n in enumerate(c.lens):
        nq = new[s]
        old = stored(before, c.table[s], n, 0, c.d)
        for j in range(nq):
            if path[s, j] < 0:
                break
            to, at = n - nq + j, n - nq + int(path[s, j])
            if missing not in (c.table[s, to // PAGE], c.table[s, at // PAGE]):
                _put(want[c.table[s, to // PAGE], 0], to % PAGE, [part[at] for part in old], c.d)
    assert np.array_equal(want, after)


def test_move_by_paths_of_any_content_stays_within_the_cache():
    """Entries that do not ascend move something, but only slots of the path's own places."""
    lens, new, d = [300, 90], [256, 50], 64
    g = workload.rng(10)
    for _ in range(4):
        c = Paged(lens, 2, d, 72, extra=1)
        data = Guarded(c.data.shape, torch.uint8, c.data)
        path = g.integers(-3, 400, (2, 256)).astype(np.int32)
        path[:, :20] = g.integers(0, 50, (2, 20))
        path[1, 3] = 2 ** 31 - 1
        before = data.t.clone()
        nv.kv_move(nv.KvCache(data.t, 2, d, 1.0, 1.0), c.table_t, c.lens_t, starts(new), int32(path))
        torch.cuda.synchronize()
        data.check()
        changed = {int(p) for p in torch.nonzero((data.t != before).any(-1).any(-1)).flatten()}
        assert changed <= {int(c.table[s, (lens[s] - new[s] + j) // PAGE]) for s in range(2) for j in range(new[s])}


def test_descending_starts_touch_nothing_beyond_the_arrays():
    c = Paged([300, 90, 64], 1, 64, 73)
    total, max_q = 60, 24
    g = workload.rng(11)
    for order in ([total, 0, 20, 40], [7, 3, total, 0], [-5, 90, 10, 10 ** 9]):
        parents, st = int32(_tree_case(g, [total], total, 0.3)), int32(order)
        masks, positions = Guarded((total, 1), torch.int64), Guarded((total,), torch.int32)
        nv.kv_tree(parents, c.lens_t, st, max_q, masks=masks.t, positions=positions.t)
        outs = [Guarded(shape, torch.int32) for shape in ((3, max_q), (3,), (3,), (3,))]
        nv.tree_accept(int32(g.integers(0, 2, total)), parents, int32(g.integers(0, 2, total)), c.lens_t, st, max_q, path=outs[0].t,
                       counts=outs[1].t, token=outs[2].t, new_lens=outs[3].t)
        data = Guarded(c.data.shape, torch.uint8, c.data)
        nv.kv_move(nv.KvCache(data.t, 1, 64, 1.0, 1.0), c.table_t, c.lens_t, st, outs[0].t)
        torch.cuda.synchronize()
        for x in (masks, positions, data, *outs):
            x.check()

"""Trees over caches of so few pages that a workgroup of the tiles takes a segment
whole (gpu), against the float64 oracle.  Tolerances are test_gpu_kv.py's."""
import numpy as np
import pytest

import workload
from tests._kv import Paged
from tests.test_gpu_kv import _query_bits
from tests.test_gpu_tree_attention import _attend, _check, _of_trees

pytestmark = pytest.mark.gpu


# up to 64 sequences each wavefront adds up the sizes, more a kernel before; tiles of 64 rows and of 128
@pytest.mark.parametrize("seqs,window", [(60, 0), (65, 0), (60, 3), (64, 60), (65, 60)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_whole_segments(seqs, d, window):
    g, group = workload.rng(91), 8
    longest = 250 if window == 0 else 900                    # under a window, 4 pages of any length
    most = 256 if window == 0 else 128
    lens = [int(g.integers(1, longest)) for _ in range(seqs)]
    new = [min(n, int(g.integers(1, 60))) for n in lens]
    lens[3], new[3] = 0, 0                                   # nothing at all
    new[7] = 0                                               # no nodes
    lens[8], new[8] = 0, 2                                   # nodes without a slot
    lens[9], new[9] = 1, 1
    lens[-1], new[-1] = longest, min(longest, most)
    c = Paged(lens, 8, d, 92)
    masks, positions = _of_trees(g, lens, new, near=3)
    qb = _query_bits(sum(new), 8 * group, d, 93)
    out, lse = _attend(c, qb, new, masks, positions, max_q=most, window=window)
    some = [0, 3, 7, 8, 9, 20, seqs - 1]
    at = np.concatenate([[0], np.cumsum(new)])
    rows = np.concatenate([np.arange(at[s], at[s + 1]) for s in some])
    heads = slice(0, 8 * group, 7)                           # a query head of each kv head is looked at
    few = type("Few", (), dict(lens=[lens[s] for s in some], d=d, heads=len(range(0, 8 * group, 7)),
                               k=[[c.k[s][h // group] for h in range(0, 8 * group, 7)] for s in some],
                               v=[[c.v[s][h // group] for h in range(0, 8 * group, 7)] for s in some]))
    _check(few, qb[rows][:, heads], [new[s] for s in some], [masks[r] for r in rows], [positions[r] for r in rows], out[rows][:, heads],
           lse[rows][:, heads], window=window)
    seen = np.ones(sum(new), bool)
    seen[at[8]:at[9]] = False
    assert np.isfinite(out).all() and np.isfinite(lse[seen]).all() and np.isneginf(lse[~seen]).all() and not out[~seen].any()


def test_tiles_of_64_rows_take_segments_whole():
    g = workload.rng(94)
    lens = [int(g.integers(10, 250)) for _ in range(64)]
    new = [int(g.integers(1, 9)) for _ in lens]
    c = Paged(lens, 64, 64, 95)
    masks, positions = _of_trees(g, lens, new)
    qb = _query_bits(sum(new), 512, 64, 96)
    out, lse = _attend(c, qb, new, masks, positions, max_q=8)
    some, at = [0, 31, 63], np.concatenate([[0], np.cumsum(new)])
    rows = np.concatenate([np.arange(at[s], at[s + 1]) for s in some])
    few = type("Few", (), dict(lens=[lens[s] for s in some], d=64, heads=64, k=[c.k[s] for s in some], v=[c.v[s] for s in some]))
    _check(few, qb[rows], [new[s] for s in some], [masks[r] for r in rows], [positions[r] for r in rows], out[rows], lse[rows])
    assert np.isfinite(out).all() and np.isfinite(lse).all()

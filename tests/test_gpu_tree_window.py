"""Windows that are shorter than drafted trees (gpu), against the float64 oracle.

Tolerances are those of test_gpu_kv.py, which derives them: the arithmetic is the
same, only what a row sees differs."""
import numpy as np
import pytest

import workload
from oracle import bf16_bits_to_f64
from oracle import draft as odraft
from tests._kv import Paged
from tests.test_gpu_kv import _check as check_causal
from tests.test_gpu_kv import _eps, _query_bits
from tests.test_gpu_tree_attention import _attend, _of_trees

pytestmark = pytest.mark.gpu


def _check(c, qbits, new, masks, positions, out, lse, window, whole_tree):
    q, at = bf16_bits_to_f64(qbits), 0
    for s, n in enumerate(c.lens):
        rows = slice(at, at + new[s])
        seen = odraft.visible(n, masks[rows], positions[rows], window, whole_tree)
        for h in range(q.shape[1]):
            k, v = c.k[s][h // (q.shape[1] // c.heads)], c.v[s][h // (q.shape[1] // c.heads)]
            o, l, spread, size = odraft.attention(q[rows, h], k, v, seen, c.d ** -0.5)
            eps = _eps(size, c.d, 0.0)[:, None]
            tol = 2.0 ** -8 * np.abs(o) + (eps + 2.0 ** -10) * spread + (n + 1) * 2.0 ** -24 * np.abs(v).max()
            assert np.all(np.abs(out[rows, h] - o) <= tol), (s, h)
            assert np.all(np.abs(lse[rows, h] - l) <= eps[:, 0] + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(l))), (s, h)
        at += new[s]


# up to 16, 32, 64 and more rows a kv head
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new,heads,group,d", [([1, 3], 2, 4, 128), ([9, 16], 2, 1, 64), ([60, 30], 1, 2, 128), ([64, 33], 1, 1, 64),
                                               ([100, 130], 1, 1, 256), ([256, 65], 1, 1, 64)])
def test_a_chain_sees_what_causal_attention_sees(new, heads, group, d, wide):
    lens = [700, 130]
    c = Paged(lens, heads, d, 14)
    masks = [(2 << i) - 1 for n in new for i in range(n)]
    positions = [n - nq + i for n, nq in zip(lens, new) for i in range(nq)]
    qb = _query_bits(sum(new), heads * group, d, 15)
    for window in (1, 8, 63, 64, 100):
        out, lse = _attend(c, qb, new, masks, positions, wide=wide, window=window)
        check_causal(c, qb, new, out, lse, window=window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new,group,d", [([12, 40], 1, 128), ([64, 33], 1, 64), ([130, 256], 1, 64), ([70, 9], 1, 256)])
def test_deep_trees(new, group, d, wide):
    # each node mostly continues one of the last two; and masks that say all that is seen of a tree
    lens = [300, 256]
    c = Paged(lens, 1, d, 500 + d)
    masks, positions = _of_trees(workload.rng(61), lens, new, near=2)
    qb = _query_bits(sum(new), group, d, 5)
    for window in (1, 5):
        seen = {}
        for whole in (False, True):
            out, seen[whole] = _attend(c, qb, new, masks, positions, window=window, wide=wide, whole_tree=whole)
            _check(c, qb, new, masks, positions, out, seen[whole], window, whole)
        assert not np.array_equal(seen[False], seen[True])

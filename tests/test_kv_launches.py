"""Calls of more workgroups than one launch has threads for: the numbers on the CPU,
the calls themselves against the oracle (gpu)."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_workgroups_at_the_ends_of_every_field(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    out = str(tmp_path / "kv_launch_check")
    host = os.path.join(ROOT, "verify_nvfp4_w4a16_amd", "csrc", "host")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "kv_launch_check.cpp"),
           *(os.path.join(host, n) for n in ("kv_shapes.cpp", "draft_shapes.cpp", "kv_plan.cpp", "tree_plan.cpp")), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "launches ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])


def _same(out, lse, rows, sequences):
    """Whether the rows of all these sequences have the first one's bits."""
    o, l = out[:sequences * rows].view(sequences, rows, -1), lse[:sequences * rows].view(sequences, rows, -1)
    return bool((o == o[:1]).all()) and bool((l == l[:1]).all())


@pytest.mark.gpu
def test_join_of_more_rows_than_a_launch_has_threads_for():
    # trees of 32 nodes and 32 heads: 2^19 (token, sequence) rows of short caches, then a tree over a cache of two parts,
    # whose rows are those from 2^24 on
    import torch

    import verify_nvfp4_w4a16_amd as nv
    import workload
    from tests._kv import Paged, bf16, int32, starts
    from tests.test_gpu_kv import _query_bits
    from tests.test_gpu_tree_attention import _check, _masks, _of_trees
    lens, nodes, heads, many = [70, 2100], 32, 32, 16384
    c = Paged(lens, heads, 64, 71)
    masks, _ = _of_trees(workload.rng(72), lens, [nodes, nodes])
    total = (many + 1) * nodes
    assert total * heads > 1 << 24
    qb = _query_bits(2 * nodes, heads, 64, 73)
    ends = bf16(qb)
    q = torch.cat([ends[:nodes].repeat(many, 1, 1), ends[nodes:]])
    m = _masks(masks, 1)
    m = torch.cat([m[:nodes].repeat(many, 1), m[nodes:]])
    table = torch.cat([c.table_t[:1].repeat(many, 1), c.table_t[1:]])
    out, lse = nv.kv_tree_attention(q, c.cache, table, int32([lens[0]] * many + [lens[1]]), starts([nodes] * (many + 1)), m, None, nodes,
                                    lens[1])
    pick = torch.cat([torch.arange(nodes), torch.arange(total - nodes, total)]).to(out.device)
    _check(c, qb, [nodes, nodes], masks, None, out[pick].float().cpu().numpy().astype(np.float64), lse[pick].cpu().numpy().astype(np.float64))
    assert _same(out, lse, nodes, many)


@pytest.mark.gpu
def test_more_single_tokens_than_a_launch_has_threads_for():
    import torch

    import verify_nvfp4_w4a16_amd as nv
    from tests._kv import Paged, bf16, int32, starts
    from tests.test_gpu_kv import _check, _query_bits
    heads, many = 257, 65535
    assert heads * many > 1 << 24
    c = Paged([3, 60], heads, 64, 74)
    qb = _query_bits(2, heads, 64, 75)
    ends = bf16(qb)
    q = torch.cat([ends[:1].expand(many - 1, heads, 64), ends[1:]])
    table = torch.cat([c.table_t[:1].repeat(many - 1, 1), c.table_t[1:]])
    out, lse = nv.kv_attention(q, c.cache, table, int32([3] * (many - 1) + [60]), starts([1] * many), 1, 60)
    _check(c, qb, [1, 1], out[[0, many - 1]].float().cpu().numpy().astype(np.float64), lse[[0, many - 1]].cpu().numpy().astype(np.float64))
    assert _same(out, lse, 1, many - 1)


@pytest.mark.gpu
def test_a_bound_on_the_new_tokens_far_above_them():
    # 2^24 tokens of 129 heads would be more workgroups than a launch has threads for
    import torch

    import verify_nvfp4_w4a16_amd as nv
    from tests._kv import Paged, bf16, starts
    from tests.test_gpu_kv import _check, _query_bits
    c, new = Paged([200, 90], 129, 64, 76), [100, 40]
    qb = _query_bits(140, 129, 64, 77)
    out, lse = nv.kv_attention(bf16(qb), c.cache, c.table_t, c.lens_t, starts(new), 1 << 24, 200)
    torch.cuda.synchronize()
    _check(c, qb, new, out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64))


@pytest.mark.gpu
def test_append_and_read_of_more_tokens_than_a_launch_has_threads_for():
    # of 65535 sequences the first and the last have a page; the others' tokens are dropped, and read as zeros
    import torch

    import verify_nvfp4_w4a16_amd as nv
    from tests._kv import DEV, bf16, int32, starts
    from tests.test_gpu_kv import _query_bits
    heads, many, d = 129, 65535, 256
    rows = bf16(_query_bits(2, heads, d, 78))
    want = nv.KvCache.empty(2, heads, d, 2.0 ** -6, 2.0 ** -7)
    nv.kv_append(want, rows, rows.flip(0).contiguous(), int32([[0], [1]]), int32([1, 1]), starts([1, 1]))
    want_k, want_v = nv.kv_read(want, int32([[0], [1]]), int32([1, 1]), starts([1, 1]), 2)
    got = nv.KvCache.empty(2, heads, d, 2.0 ** -6, 2.0 ** -7)
    table = torch.full((many, 1), -1, dtype=torch.int32, device=DEV)
    table[0, 0], table[-1, 0] = 0, 1
    where = (table, int32([1] * many), starts([1] * many))
    k, v = (torch.ones((many, heads, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[0], k[-1], v[0], v[-1] = rows[0], rows[1], rows[1], rows[0]
    nv.kv_append(got, k, v, *where)
    assert torch.equal(got.data, want.data)
    nv.kv_read(got, *where, many, k=k, v=v)
    for x, y in ((k, want_k), (v, want_v)):
        assert torch.equal(x[0], y[0]) and torch.equal(x[-1], y[1]) and not bool(x[1:-1].any())


@pytest.mark.gpu
def test_slot_weights_under_the_largest_bound_on_the_slots():
    import torch

    import verify_nvfp4_w4a16_amd as nv
    from tests._kv import DEV, Paged, bf16, starts
    from tests.test_gpu_kv import _query_bits
    heads, new, pitch = 8, 130, 1 << 23
    c = Paged([150], heads, 64, 79)
    q, st = bf16(_query_bits(new, heads, 64, 80)), starts([new])
    _, lse = nv.kv_attention(q, c.cache, c.table_t, c.lens_t, st, new, 150)
    want = nv.kv_weights(q, lse, c.cache, c.table_t, c.lens_t, st, new, 150)
    table = torch.full((1, pitch), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table_t.shape[1]] = c.table_t
    got = torch.ones((1, heads, pitch * 64), dtype=torch.float32, device=DEV)
    nv.kv_weights(q, lse, c.cache, table, c.lens_t, st, new, pitch * 64, out=got)
    # few pages are shared by a workgroup's wavefronts, many are not: sums of the same 130 numbers, none negative, in two
    # orders, each with at most 130 roundings of half a step, 2^-24 of a sum that is no larger than the last
    assert torch.allclose(got[..., :150], want, rtol=2 * new * 2.0 ** -24, atol=0)
    assert not any(bool(got[0, h, 150:].any()) for h in range(heads))


@pytest.mark.gpu
def test_eviction_to_a_bound_far_above_the_slots():
    import torch

    import verify_nvfp4_w4a16_amd as nv
    from tests._kv import DEV, Paged, int32
    heads, n, d = 64, 150, 256
    c = Paged([n], heads, d, 81)
    w = torch.rand((1, heads, n), device=DEV)
    made = []
    for keep in (192, (1 << 23) + 64):
        dst = nv.KvCache.empty(3, heads, d, c.k_scale, c.v_scale)
        table = torch.full((1, keep // 64), -1, dtype=torch.int32, device=DEV)
        table[0, :3] = int32([2, 0, 1])
        kept, weights, lens = nv.kv_evict(w, c.cache, c.table_t, c.lens_t, table, keep, dst=dst)
        made.append((dst.data, kept[..., :192], weights[..., :192], lens))
        assert bool((kept[..., n:] == -1).all()) and not bool(weights[..., n:].any())
    for a, b in zip(*made):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_more_trees_in_tiles_than_a_launch_has_threads_for():
    # a bound of 33 nodes makes it a call for the tiles, of whole segments
    import torch

    import verify_nvfp4_w4a16_amd as nv
    from tests._kv import Paged, bf16, int32, starts
    from tests.test_gpu_kv import _query_bits
    from tests.test_gpu_tree_attention import _check
    heads, many = 257, 65535
    c = Paged([3, 60], heads, 64, 82)
    qb = _query_bits(2, heads, 64, 83)
    ends = bf16(qb)
    q = torch.cat([ends[:1].expand(many - 1, heads, 64), ends[1:]])
    table = torch.cat([c.table_t[:1].repeat(many - 1, 1), c.table_t[1:]])
    masks = torch.ones((many, 1), dtype=torch.int64, device=q.device)
    out, lse = nv.kv_tree_attention(q, c.cache, table, int32([3] * (many - 1) + [60]), starts([1] * many), masks, None, 33, 60)
    _check(c, qb, [1, 1], [1, 1], None, out[[0, many - 1]].float().cpu().numpy().astype(np.float64),
           lse[[0, many - 1]].cpu().numpy().astype(np.float64))
    assert _same(out, lse, 1, many - 1)

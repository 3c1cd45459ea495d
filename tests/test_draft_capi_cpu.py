"""Host side of the verify round's C ABI, on the CPU: exports, constants, the
refusals (every argument is checked before any GPU call), the checks under
sanitizers, and the oracle the GPU tests compare with, pinned to closed forms.
No GPU call is made here."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import verify_nvfp4_w4a16_amd as nv
from oracle import draft as odraft
from oracle import kv as okv

torch = pytest.importorskip("torch")
from tests.test_kv_capi_cpu import A, BAD_CACHE, BAD_QUERIES, BAD_SEQS, _cache, _queries, _seqs  # noqa: E402
from tests.test_kv_refusals import _host_cache  # noqa: E402
from verify_nvfp4_w4a16_amd import drafting  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_draft.h")


def test_library_exports_every_declared_function():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"^int (nvfp4_\w+)\(", text, re.M)))
    assert declared == sorted(drafting.EXPORTED)
    lib = ctypes.CDLL(nv.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name
    for name, value in (("NVFP4_TREE_MAX", drafting.TREE_MAX), ("NVFP4_TREE_WORDS", drafting.TREE_WORDS), ("NVFP4_BIAS_MAX", drafting.BIAS_MAX)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value


def test_names_are_the_package_s():
    for name in nv._DRAFTING:
        assert getattr(nv, name) is getattr(drafting, name)


def test_checks_at_the_ends_of_every_field(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    out = str(tmp_path / "draft_host_check")
    host = os.path.join(ROOT, "verify_nvfp4_w4a16_amd", "csrc", "host")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "draft_host_check.cpp"),
           os.path.join(host, "kv_shapes.cpp"), os.path.join(host, "draft_shapes.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "host ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])


def test_refusals_of_pages():
    lib = drafting._draft()

    def call(state_out=A, held_out=A, kv_lens=A, q_starts=A, slots=A, positions=A, **kw):
        f = dict(pool=A, state=A, capacity=10, table=A, table_pitch=4, held=A, keep=A, fresh=A, seqs=2, total=8)
        f.update(kw)
        return lib.nvfp4_kv_pages(drafting._Pages(*f.values()), state_out, held_out, kv_lens, q_starts, slots, positions, None)

    for kw in (dict(capacity=0), dict(capacity=(1 << 30) + 1), dict(table_pitch=0), dict(table_pitch=(1 << 23) + 1), dict(seqs=-1),
               dict(seqs=65536), dict(total=-1), dict(total=(1 << 24) + 1)):
        assert call(**kw) == nv.ERR_SHAPE, kw
    # pages of a block of sequences that would not add up in 32 bits, whatever `held` says
    for kw in (dict(seqs=129, table_pitch=1 << 23), dict(seqs=1024, table_pitch=(1 << 20) + 1), dict(seqs=65535, table_pitch=(1 << 20) + 1)):
        assert call(**kw) == nv.ERR_SHAPE, kw
    for name in ("pool", "state", "table", "held", "keep", "fresh", "state_out", "held_out", "kv_lens", "q_starts"):
        assert call(**{name: None}) == nv.ERR_NULL, name
        assert call(**{name: A + 2}) == nv.ERR_ALIGN, name
    for name in ("slots", "positions"):
        assert call(**{name: A + 1}) == nv.ERR_ALIGN, name
    assert lib.nvfp4_kv_pages(None, A, A, A, A, A, A, None) == nv.ERR_NULL


def test_refusals_of_trees():
    lib = drafting._draft()

    def tree(parents=A, kv_lens=A, q_starts=A, seqs=2, total=8, max_q=4, masks=A, positions=A):
        return lib.nvfp4_kv_tree(parents, kv_lens, q_starts, seqs, total, max_q, masks, positions, None)

    def accept(drafted=A, parents=A, chosen=A, kv_lens=A, q_starts=A, seqs=2, total=8, max_q=4, path=A, counts=A, token=A, new_lens=A):
        return lib.nvfp4_tree_accept(drafted, parents, chosen, kv_lens, q_starts, seqs, total, max_q, path, counts, token, new_lens, None)

    for call in (tree, accept):
        for kw in (dict(seqs=-1), dict(seqs=65536), dict(total=-1), dict(total=(1 << 24) + 1), dict(max_q=0), dict(max_q=257)):
            assert call(**kw) == nv.ERR_SHAPE, kw
        assert call(seqs=0, kv_lens=None) == nv.OK
    for call, names in ((tree, ("parents", "kv_lens", "q_starts", "masks", "positions")),
                        (accept, ("drafted", "parents", "chosen", "kv_lens", "q_starts", "path", "counts", "token", "new_lens"))):
        for name in names:
            assert call(**{name: None}) == nv.ERR_NULL, name
            assert call(**{name: A + 2}) == nv.ERR_ALIGN, name
    assert tree(masks=A + 4) == nv.ERR_ALIGN
    assert tree(total=0, parents=None, masks=None, positions=None) == nv.OK


def _tree(**kw):
    f = dict(masks=A, positions=A, words=1)
    f.update(kw)
    return drafting._Tree(*f.values())


def test_refusals_of_tree_attention():
    lib = drafting._draft()
    c, s, q = _cache(), _seqs(), _queries()

    def call(c=c, s=s, q=q, t=_tree(), out=A, lse=A, ws=A, wb=1 << 40):
        return lib.nvfp4_kv_tree_attention(c, s, q, t, out, lse, ws, wb, None)

    for kw, want in BAD_CACHE:
        assert call(c=_cache(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        assert call(s=_seqs(**kw)) == want, kw
    for kw, want in BAD_QUERIES:
        assert call(q=_queries(**kw)) == want, kw
        assert lib.nvfp4_kv_tree_attention_workspace(c, s, _queries(**kw), ctypes.c_int64()) == want, kw
    assert call(t=None) == nv.ERR_NULL
    for kw, want in ((dict(masks=0), nv.ERR_NULL), (dict(masks=A + 4), nv.ERR_ALIGN), (dict(positions=A + 2), nv.ERR_ALIGN),
                     (dict(words=0), nv.ERR_SHAPE), (dict(words=5), nv.ERR_SHAPE)):
        assert call(t=_tree(**kw)) == want, kw
    assert call(q=_queries(max_q=65)) == nv.ERR_SHAPE
    assert call(q=_queries(max_q=257), t=_tree(words=4)) == nv.ERR_SHAPE
    assert call(q=_queries(window=5), t=_tree(positions=0)) == nv.ERR_NULL
    assert call(out=None) == nv.ERR_NULL and call(out=A + 2) == nv.ERR_ALIGN and call(lse=A + 2) == nv.ERR_ALIGN
    need = ctypes.c_int64()
    wide, long = _seqs(table_pitch=2048), _queries(max_kv=128 * 1024)
    assert lib.nvfp4_kv_tree_attention_workspace(c, wide, long, need) == nv.OK and need.value > 0
    assert call(s=wide, q=long, wb=need.value - 1) == nv.ERR_SCRATCH
    assert call(s=wide, q=long, ws=None) == nv.ERR_NULL
    assert lib.nvfp4_kv_tree_attention_workspace(c, s, q, None) == nv.ERR_NULL


def test_refusals_of_adjust():
    lib = drafting._draft()

    def call(out=A, **kw):
        f = {name: 0 for name, _ in drafting._Adjust._fields_}
        f.update(logits=A, rows=2, vocab=100, pitch=100, out_pitch=100, logits_type=1, out_type=1, seqs=2)
        f.update(kw)
        return lib.nvfp4_adjust_logits(drafting._Adjust(*f.values()), out, None)

    for kw in (dict(rows=-1, seqs=-1), dict(rows=65536, seqs=65536), dict(vocab=0), dict(vocab=(1 << 22) + 1, pitch=1 << 23, out_pitch=1 << 23),
               dict(pitch=99), dict(out_pitch=99), dict(seqs=3), dict(history=A, history_lens=A, history_pitch=(1 << 19) + 1),
               dict(history=A, history_lens=A, history_pitch=-1), dict(bias_tokens=A, bias_values=A, bias_width=1025),
               dict(allowed=A, allowed_pitch=3, states=2), dict(allowed=A, allowed_pitch=4, states=-1),
               dict(drafted=A, masks=A, mask_words=0), dict(drafted=A, masks=A, mask_words=5), dict(out_pitch=101), dict(out_type=0)):
        assert call(**kw) == nv.ERR_SHAPE, kw
    assert call(logits_type=2) == nv.ERR_DTYPE and call(out_type=-1) == nv.ERR_DTYPE
    for kw in (dict(logits=0), dict(history=A), dict(bias_tokens=A, bias_width=3), dict(drafted=A, mask_words=1)):
        assert call(**kw) == nv.ERR_NULL, kw
    assert call(out=None) == nv.ERR_NULL
    for kw in (dict(logits=A + 2), dict(logits=A + 1, logits_type=0, out_type=0), dict(q_starts=A + 2), dict(history=A + 2, history_lens=A),
               dict(history=A, history_lens=A + 2), dict(prompt_lens=A + 1), dict(repetition=A + 2), dict(presence=A + 2),
               dict(frequency=A + 2), dict(bias_tokens=A + 2, bias_values=A, bias_width=3), dict(bias_tokens=A, bias_values=A + 1, bias_width=3),
               dict(allowed=A + 2, allowed_pitch=4, states=2), dict(allowed_rows=A + 2), dict(drafted=A + 2, masks=A, mask_words=1),
               dict(drafted=A, masks=A + 4, mask_words=1)):
        assert call(**kw) == nv.ERR_ALIGN, kw
    assert call(out=A + 2) == nv.ERR_ALIGN
    assert call(rows=0, seqs=0, logits=0, out=None) == nv.OK
    assert lib.nvfp4_adjust_logits(None, A, None) == nv.ERR_NULL


def test_refusals_of_move():
    lib = drafting._draft()
    far = 1 << 30

    def call(*caches, s=None, path=A, max_q=4, count=None):
        caches = caches or (_cache(), _cache(data=far))
        n = len(caches) if count is None else count
        return lib.nvfp4_kv_move((drafting._Cache * len(caches))(*caches), n, s or _seqs(), path, max_q, None)

    for kw, want in BAD_CACHE:
        assert call(_cache(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        assert call(s=_seqs(**kw)) == want, kw
    for kw in (dict(head_dim=64), dict(kv_heads=1), dict(pages=5)):
        assert call(_cache(), _cache(data=far, **kw)) == nv.ERR_SHAPE, kw
    # the same data twice, or data that overlap
    assert call(_cache(), _cache()) == nv.ERR_SHAPE
    assert call(_cache(), _cache(data=far), _cache(data=A + 16)) == nv.ERR_SHAPE
    assert call(count=0) == nv.ERR_SHAPE and call(max_q=0) == nv.ERR_SHAPE and call(max_q=257) == nv.ERR_SHAPE
    assert call(path=None) == nv.ERR_NULL and call(path=A + 2) == nv.ERR_ALIGN
    assert lib.nvfp4_kv_move(None, 1, _seqs(), A, 4, None) == nv.ERR_NULL


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_python_refuses_wrong_tensors():
    cache = _host_cache()
    with pytest.raises(ValueError):                                            # not on a GPU
        nv.kv_pages(_i32(4), _i32(2), _i32(2, 3), _i32(2), _i32(2), _i32(2), 4)
    with pytest.raises(ValueError):
        nv.kv_tree(_i32(4), _i32(1), _i32(2), 4)
    with pytest.raises(ValueError):
        nv.tree_accept(_i32(4), _i32(4), _i32(4), _i32(1), _i32(2), 4)
    with pytest.raises(ValueError):
        nv.adjust_logits(torch.zeros(2, 10))
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    where = (cache, _i32(1, 1), _i32(1), _i32(2))
    for masks in (torch.zeros(4, dtype=torch.int64), _i32(4, 1), torch.zeros(3, 1, dtype=torch.int64),
                  torch.zeros(4, 2, dtype=torch.int64)[:, ::2], torch.zeros(4, 1, dtype=torch.int64, device="meta")):
        with pytest.raises(ValueError):
            nv.kv_tree_attention(q, *where, masks, None, 4, 4)
    masks = torch.zeros(4, 1, dtype=torch.int64)
    for positions in (_i32(3), torch.zeros(4), _i32(8)[::2]):
        with pytest.raises(ValueError):
            nv.kv_tree_attention(q, *where, masks, positions, 4, 4)
    with pytest.raises(ValueError):
        nv.kv_move([], *where[1:], _i32(1, 4))
    with pytest.raises(ValueError):
        nv.kv_move([cache, _host_cache("meta")], *where[1:], _i32(1, 4))
    for path in (_i32(4), _i32(2, 4), torch.zeros(1, 4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            nv.kv_move(cache, *where[1:], path)


# ---- the oracle

def test_oracle_pages_closed_forms():
    # pool: pages 7, 8, 9 from entry 3 of 5 on (9 lies at the front); one sequence grows, one ends, one is refused
    pool, state, table, held, lens, starts, slots, positions = odraft.pages(
        [9, 0, 0, 7, 8], [3, 3], [[5, -1], [6, -1], [4, -1]], [1, 1, 1], [64, 0, 64], [2, 0, 200], 10)
    assert pool == [9, 6, 0, 7, 8] and state == [4, 3]        # one page came from the front, page 6 went to the back
    assert table.tolist() == [[5, 7], [6, -1], [4, -1]] and held == [2, 0, 1] and lens == [66, 0, 64]
    assert starts == [0, 2, 2, 2] and slots == [7 * 64, 7 * 64 + 1] + [-1] * 8 and positions[:3] == [64, 65, -1]
    # what an earlier sequence asks for counts, granted or not; one that needs no page is still served
    _, state, _, held, lens, _, _, _ = odraft.pages([1, 2], [0, 2], [[0, -1, -1], [3, -1, -1], [4, -1, -1]], [1, 1, 1], [64, 64, 1],
                                                    [65, 100, 5], 300)
    assert held == [3, 1, 1] and lens == [129, 64, 6] and state[1] == 0


def test_oracle_trees_closed_forms():
    assert odraft.ways([-1, 0, 0, 1, 3, 9, 5]) == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [5], [5, 6]]
    assert odraft.mask_words([0, 63, 64], 2) == [(1 << 63) + 1, 1]
    assert odraft.accept([5, 6, 6, 7], [-1, 0, 0, 2], [6, 7, 7, 9]) == ([0, 1], 7)      # the lower of equal drafts
    assert odraft.accept([5, -1], [-1, 0], [-1, 3]) == ([0], -1)                        # no token matches none
    # a chain's masks are the causal mask
    n, nq = 9, 4
    masks = [sum(1 << a for a in w) for w in odraft.ways([-1, 0, 1, 2])]
    for window in (0, 1, 3, 6):
        seen = odraft.visible(n, masks, range(n - nq, n), window)
        chain = okv.visible(n, nq, True, window)
        before = n - nq
        assert np.array_equal(seen[:, :before], chain[:, :before]) and np.array_equal(seen[:, before:], okv.visible(n, nq, True, 0)[:, before:])
    assert odraft.visible(2, masks, None, 0).tolist() == [[False, False], [False, False], [True, False], [True, True]]


def test_oracle_ways_masks_and_branches():
    assert odraft.ways([-1, 0, 0, 1, 3, 9, 5]) == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [5], [5, 6]]
    assert odraft.mask_words([0, 63, 64], 2) == [(1 << 63) + 1, 1]
    assert odraft.accept([5, 6, 6, 7], [-1, 0, 0, 2], [6, 7, 7, 9]) == ([0, 1], 7)      # the lower of equal drafts
    assert odraft.accept([5, -1], [-1, 0], [-1, 3]) == ([0], -1)                        # no token matches none
    masks, _ = _chain(9, 4)
    assert odraft.visible(2, masks, None, 0).tolist() == [[False, False], [False, False], [True, False], [True, True]]


def _chain(n, nq):
    return [(2 << i) - 1 for i in range(nq)], list(range(n - nq, n))


@pytest.mark.parametrize("n,nq", [(9, 4), (90, 60), (64, 64), (130, 70), (1, 1), (3, 8)])
def test_oracle_chain_under_a_window_sees_what_attention_sees(n, nq):
    masks, positions = _chain(n, nq)
    for window in (0, 1, 2, 3, 6, 8, nq - 1, nq, nq + 1, n, n + 5):
        want = okv.visible(n, nq, True, window) if n >= nq else None
        seen = odraft.visible(n, masks, positions, window)
        if want is None:                       # nodes without a slot of their own see nothing, the others at most `window`
            want = np.array([[j <= n - nq + i and (not window or j > n - nq + i - window) for j in range(n)] for i in range(nq)])
        assert np.array_equal(seen, want), window


def test_oracle_windows_in_trees():
    # node 4's way is 0, 1, 3, at positions 5, 6, 7; 2 is 1's sibling
    ways = odraft.ways([-1, 0, 0, 1, 3])
    masks, positions = [sum(1 << a for a in w) for w in ways], [5 + len(w) - 1 for w in ways]
    for window, first in ((1, [8]), (2, [7, 8]), (3, [6, 7, 8]), (4, [5, 6, 7, 8]), (5, [4, 5, 6, 7, 8])):
        of = {5: 0, 6: 1, 7: 3, 8: 4}          # the node of 4's way at each position
        want = [p if p < 5 else 5 + of[p] for p in first]
        assert np.flatnonzero(odraft.visible(10, masks, positions, window)[4]).tolist() == want, window
    # masks that say all of the tree: the window counts before it alone
    seen = odraft.visible(10, masks, positions, 3, whole_tree=True)
    assert np.flatnonzero(seen[4]).tolist() == [5, 6, 8, 9] and np.flatnonzero(seen[0]).tolist() == [3, 4, 5]
    # without a window both are the same, and so they are where it has room for the tree
    for window in (0, 4, 9):
        assert np.array_equal(odraft.visible(10, masks, positions, window), odraft.visible(10, masks, positions, window, True))


def test_refusals_of_a_whole_tree():
    lib, c, s, q = drafting._draft(), _cache(), _seqs(), _queries()
    for whole in (-1, 2):
        assert lib.nvfp4_kv_tree_attention(c, s, q, _tree(whole_tree=whole), A, A, A, 1 << 40, None) == nv.ERR_SHAPE


def test_oracle_attention_is_the_cache_s():
    g = np.random.default_rng(4)
    q, k, v = g.standard_normal((3, 64)), g.standard_normal((7, 64)), g.standard_normal((7, 64))
    for cap in (0.0, 2.0):
        for a, b in zip(odraft.attention(q, k, v, okv.visible(7, 3, True, 0), 0.3, cap), okv.attention(q, k, v, 0.3, True, 0, cap)):
            assert np.allclose(a, b, rtol=1e-14)


def test_oracle_adjust_closed_forms():
    x, _ = odraft.adjust([2.0, -2.0, 1.0, 3.0], [0], [1, 1, 9], r=2.0, p=0.5, f=0.25, bias=[(2, 1.0), (2, -4.0), (7, 1.0)], allowed=[1, 1, 1, 0])
    assert x.tolist() == [1.0, -5.0, -3.0, -np.inf]
    x, _ = odraft.adjust([2.0, np.nan], [0, 1], [], r=-1.0)
    assert x[0] == 2.0 and np.isnan(x[1])


def test_layout_of_tree_attention_at_the_ends_of_every_field(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    out = str(tmp_path / "tree_plan_check")
    host = os.path.join(ROOT, "verify_nvfp4_w4a16_amd", "csrc", "host")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "tree_plan_check.cpp"),
           *(os.path.join(host, n) for n in ("kv_shapes.cpp", "draft_shapes.cpp", "kv_plan.cpp", "tree_plan.cpp")), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "plan ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])


def test_a_stream_may_be_a_handle_alone(monkeypatch):
    from verify_nvfp4_w4a16_amd import serving

    class Handle:
        cuda_stream = 55

    calls = []
    monkeypatch.setattr(serving, "_current_device", lambda: 0)
    serving._launch("x", lambda *args: calls.append(args) or nv.OK, torch.device("cuda:0"), Handle, 1)
    assert calls == [(1, 55)]


def test_calls_run_with_their_tensors_device_current(monkeypatch):
    from verify_nvfp4_w4a16_amd import serving
    current, calls = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *error):
            current[0] = self.before

    class Stream:
        device, cuda_stream = torch.device("cuda:1"), 77

    monkeypatch.setattr(serving, "_current_device", lambda: current[0])
    monkeypatch.setattr(serving, "_raw_stream", lambda index: 10 + index)
    monkeypatch.setattr(serving.torch.cuda, "device", Device)

    def call(*args):
        calls.append((current[0], args))
        return nv.OK

    serving._launch("x", call, torch.device("cuda:0"), None, 1)
    serving._launch("x", call, torch.device("cuda:1"), None, 2)
    serving._launch("x", call, torch.device("cuda:1"), Stream, 3)
    assert calls == [(0, (1, 10)), (1, (2, 11)), (1, (3, 77))] and current == [0]
    with pytest.raises(ValueError, match="stream"):
        serving._launch("x", call, torch.device("cuda:0"), Stream, 4)
    assert len(calls) == 3

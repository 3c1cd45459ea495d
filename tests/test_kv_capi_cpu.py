"""Host side of the serving calls' C ABI, on the CPU: exports, constants, the
refusals (every argument is checked before any GPU call) and the oracle the GPU
tests compare with, pinned to closed forms.  No GPU call is made here."""
import ctypes
import os
import re

import numpy as np
import pytest

import oracle
import verify_nvfp4_w4a16_amd as nv
from oracle import kv as okv
from oracle.sample import sample as sample_ref

torch = pytest.importorskip("torch")
from verify_nvfp4_w4a16_amd import serving  # noqa: E402

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "nvfp4_kv.h")
A = 1 << 20            # an aligned address that no call here reaches


def test_library_exports_every_declared_function():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"^int (nvfp4_\w+)\(", text, re.M)))
    assert declared == sorted(serving.EXPORTED)
    lib = ctypes.CDLL(nv.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name
    assert int(re.search(r"#define NVFP4_KV_PAGE (\d+)", text).group(1)) == serving.PAGE == okv.PAGE
    assert int(re.search(r"NVFP4_LOGITS_BF16 = (\d)", text).group(1)) == serving.LOGITS_BF16
    assert int(re.search(r"NVFP4_LOGITS_F32 = (\d)", text).group(1)) == serving.LOGITS_F32


def test_names_are_the_package_s():
    for name in ("KvCache", "kv_append", "kv_read", "kv_attention", "kv_weights", "kv_evict", "sample"):
        assert getattr(nv, name) is getattr(serving, name)
    with pytest.raises(AttributeError):
        nv.no_such_name


def test_record_bytes():
    n = ctypes.c_int64()
    lib = serving._kv()
    for d in (64, 128, 256):
        assert lib.nvfp4_kv_record_bytes(d, n) == nv.OK and n.value == 72 * d
    assert lib.nvfp4_kv_record_bytes(96, n) == nv.ERR_SHAPE
    assert lib.nvfp4_kv_record_bytes(64, None) == nv.ERR_NULL


def _cache(**kw):
    f = dict(data=A, pages=4, kv_heads=2, head_dim=128, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return serving._Cache(*f.values())


def _seqs(**kw):
    f = dict(table=A, kv_lens=A, q_starts=A, table_pitch=2, seqs=3, total=7)
    f.update(kw)
    return serving._Seqs(*f.values())


def _queries(**kw):
    f = dict(q=A, q_pitch=1024, q_head_pitch=128, heads=8, max_q=4, max_kv=100, window=0, scale=0.1, softcap=0.0, causal=1)
    f.update(kw)
    return serving._Queries(*f.values())


BAD_CACHE = [(dict(data=0), nv.ERR_NULL), (dict(data=A + 8), nv.ERR_ALIGN), (dict(pages=-1), nv.ERR_SHAPE),
             (dict(kv_heads=0), nv.ERR_SHAPE), (dict(kv_heads=1025), nv.ERR_SHAPE), (dict(head_dim=96), nv.ERR_SHAPE),
             (dict(k_scale=0.0), nv.ERR_SHAPE), (dict(v_scale=float("nan")), nv.ERR_SHAPE),
             (dict(k_scale=float("inf")), nv.ERR_SHAPE), (dict(v_scale=-1.0), nv.ERR_SHAPE)]
BAD_SEQS = [(dict(table=0), nv.ERR_NULL), (dict(kv_lens=0), nv.ERR_NULL), (dict(q_starts=0), nv.ERR_NULL),
            (dict(table=A + 2), nv.ERR_ALIGN), (dict(kv_lens=A + 1), nv.ERR_ALIGN), (dict(q_starts=A + 2), nv.ERR_ALIGN),
            (dict(table_pitch=0), nv.ERR_SHAPE), (dict(table_pitch=(1 << 23) + 1), nv.ERR_SHAPE),
            (dict(seqs=-1), nv.ERR_SHAPE), (dict(seqs=65536), nv.ERR_SHAPE), (dict(total=-1), nv.ERR_SHAPE),
            (dict(total=(1 << 24) + 1), nv.ERR_SHAPE)]
BAD_QUERIES = [(dict(q=0), nv.ERR_NULL), (dict(q=A + 8), nv.ERR_ALIGN), (dict(q_pitch=1023), nv.ERR_ALIGN),
               (dict(q_head_pitch=4), nv.ERR_ALIGN), (dict(q_pitch=-8), nv.ERR_SHAPE), (dict(heads=7), nv.ERR_SHAPE),
               (dict(heads=0), nv.ERR_SHAPE), (dict(heads=2 * 257), nv.ERR_SHAPE), (dict(max_q=-1), nv.ERR_SHAPE),
               (dict(max_kv=-1), nv.ERR_SHAPE), (dict(max_kv=129), nv.ERR_SHAPE), (dict(window=-1), nv.ERR_SHAPE),
               (dict(scale=float("nan")), nv.ERR_SHAPE), (dict(softcap=-1.0), nv.ERR_SHAPE),
               (dict(softcap=float("inf")), nv.ERR_SHAPE), (dict(softcap=float("nan")), nv.ERR_SHAPE),
               (dict(causal=2), nv.ERR_SHAPE), (dict(max_q=1 << 24, heads=512), nv.ERR_SHAPE)]


def test_refusals_of_the_cache_and_the_sequences():
    lib = serving._kv()
    calls = [lambda c, s: lib.nvfp4_kv_append(c, s, A, 256, 128, A, 256, 128, None),
             lambda c, s: lib.nvfp4_kv_read(c, s, A, A, None),
             lambda c, s: lib.nvfp4_kv_attention(c, s, _queries(), A, A, A, 1 << 40, None),
             lambda c, s: lib.nvfp4_kv_attention_workspace(c, s, _queries(), ctypes.c_int64()),
             lambda c, s: lib.nvfp4_kv_weights(c, s, _queries(), A, A, A, None)]
    for call in calls:
        for kw, want in BAD_CACHE:
            assert call(_cache(**kw), _seqs()) == want, kw
        for kw, want in BAD_SEQS:
            assert call(_cache(), _seqs(**kw)) == want, kw
        assert call(None, _seqs()) == nv.ERR_NULL
        assert call(_cache(), None) == nv.ERR_NULL


def test_refusals_of_the_queries_and_outputs():
    lib = serving._kv()
    c, s = _cache(), _seqs()
    for kw, want in BAD_QUERIES:
        q = _queries(**kw)
        assert lib.nvfp4_kv_attention(c, s, q, A, A, A, 1 << 40, None) == want, kw
        assert lib.nvfp4_kv_weights(c, s, q, A, A, A, None) == want, kw
        assert lib.nvfp4_kv_attention_workspace(c, s, q, ctypes.c_int64()) == want, kw
    q = _queries()
    assert lib.nvfp4_kv_attention(c, s, None, A, A, A, 1 << 40, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_attention(c, s, q, None, A, A, 1 << 40, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_attention(c, s, q, A + 2, A, A, 1 << 40, None) == nv.ERR_ALIGN
    assert lib.nvfp4_kv_attention(c, s, q, A, A + 2, A, 1 << 40, None) == nv.ERR_ALIGN
    assert lib.nvfp4_kv_attention(c, s, q, A, A, A + 4, 1 << 40, None) == nv.ERR_ALIGN
    need = ctypes.c_int64()
    long = _queries(max_kv=128 * 1024)
    wide = _seqs(table_pitch=2048)
    assert lib.nvfp4_kv_attention_workspace(c, wide, long, need) == nv.OK and need.value > 0
    assert lib.nvfp4_kv_attention(c, wide, long, A, A, A, need.value - 1, None) == nv.ERR_SCRATCH
    assert lib.nvfp4_kv_attention(c, wide, long, A, A, None, need.value, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_attention_workspace(c, wide, long, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_weights(c, s, q, None, A, A, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_weights(c, s, q, A, A, None, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_weights(c, s, q, A, A + 1, A, None) == nv.ERR_ALIGN
    for k, pitch, want in [(None, 256, nv.ERR_NULL), (A + 2, 256, nv.ERR_ALIGN), (A, 100, nv.ERR_ALIGN), (A, -8, nv.ERR_SHAPE)]:
        assert lib.nvfp4_kv_append(c, s, k, pitch, 128, A, 256, 128, None) == want
        assert lib.nvfp4_kv_append(c, s, A, 256, 128, k, pitch, 128, None) == want
    assert lib.nvfp4_kv_read(c, s, None, A, None) == nv.ERR_NULL
    assert lib.nvfp4_kv_read(c, s, A, A + 4, None) == nv.ERR_ALIGN


def test_refusals_of_evict():
    lib = serving._kv()

    def call(c=None, s=None, w=A, wp=100, keep=64, sink=1, recent=2, dst=None, table=A, pitch=1, kept=A, kw=A, nl=A):
        return lib.nvfp4_kv_evict(c or _cache(), s or _seqs(q_starts=0), w, wp, keep, sink, recent, dst or _cache(), table,
                                  pitch, kept, kw, nl, None)

    for kw, want in BAD_CACHE:
        assert call(c=_cache(**kw)) == want, kw
        assert call(dst=_cache(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        if "q_starts" not in kw:
            assert call(s=_seqs(**kw)) == want, kw
    assert call(dst=_cache(head_dim=64)) == nv.ERR_SHAPE
    assert call(dst=_cache(kv_heads=1)) == nv.ERR_SHAPE
    for kw in (dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=33, recent=32), dict(wp=-1), dict(pitch=0),
               dict(keep=65), dict(keep=(1 << 30) + 1, pitch=1 << 23)):
        assert call(**kw) == nv.ERR_SHAPE, kw
    for name in ("w", "table", "kept", "kw", "nl"):
        assert call(**{name: None}) == nv.ERR_NULL, name
        assert call(**{name: A + 2}) == nv.ERR_ALIGN, name


def test_refusals_of_sample():
    lib = serving._kv()

    def call(logits=A, kind=1, rows=2, vocab=100, pitch=100, u=A, t=A, k=A, p=A, m=A, tok=A, lp=A, ws=A, wb=1 << 40):
        return lib.nvfp4_sample(logits, kind, rows, vocab, pitch, u, t, k, p, m, tok, lp, ws, wb, None)

    for kw in (dict(rows=-1), dict(rows=65536), dict(vocab=0), dict(vocab=(1 << 22) + 1, pitch=1 << 23), dict(pitch=99)):
        assert call(**kw) == nv.ERR_SHAPE, kw
    assert call(kind=2) == nv.ERR_DTYPE
    for name in ("logits", "u", "tok"):
        assert call(**{name: None}) == nv.ERR_NULL, name
    for name in ("logits", "u", "t", "k", "p", "m", "tok", "lp"):
        assert call(**{name: A + 2}) == nv.ERR_ALIGN, name
    assert call(logits=A + 1, kind=0) == nv.ERR_ALIGN
    assert call(rows=0, logits=None) == nv.OK
    n = ctypes.c_int64()
    assert lib.nvfp4_sample_workspace(2, 100, None) == nv.ERR_NULL
    assert lib.nvfp4_sample_workspace(2, 0, n) == nv.ERR_SHAPE
    assert lib.nvfp4_sample_workspace(2, 151552, n) == nv.OK
    if n.value:
        assert call(vocab=151552, pitch=151552, wb=n.value - 1) == nv.ERR_SCRATCH
        assert call(vocab=151552, pitch=151552, ws=None) == nv.ERR_NULL


def test_python_refuses_wrong_tensors():
    with pytest.raises(ValueError):
        nv.KvCache(torch.zeros(2, 1, 100, dtype=torch.uint8), 1, 64, 1.0, 1.0)
    with pytest.raises(ValueError):
        nv.KvCache(torch.zeros(2, 1, 72 * 64, dtype=torch.uint8), 1, 64, 1.0, 1.0)     # not on a GPU
    with pytest.raises(ValueError):
        nv.KvCache(torch.zeros(2, 1, 72 * 96, dtype=torch.uint8), 1, 96, 1.0, 1.0)
    with pytest.raises(ValueError):
        nv.sample(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(ValueError):
        nv.sample(torch.zeros(2, 10, dtype=torch.float16), torch.zeros(2))


# ---- the oracle

def test_oracle_record_round_trip_and_scale_order():
    g = np.random.default_rng(1)
    for d in (64, 128, 256):
        k, v = g.integers(0, 16, (2, 64, d), dtype=np.uint8)
        ks, vs = g.integers(0, 127, (2, 64, d // 16), dtype=np.uint8)
        rec = okv.build_record(k, ks, v, vs)
        for a, b in zip((k, ks, v, vs), okv.split_record(rec, d)):
            assert np.array_equal(a, b)
        # the scale bytes fill their regions exactly once
        at = sorted(okv.k_scale_index(s, i, d) for s in range(64) for i in range(d // 16))
        assert at == list(range(64 * d, 68 * d))
        at = sorted(okv.v_scale_index(s, i, d) for s in range(64) for i in range(d // 16))
        assert at == list(range(68 * d, 72 * d))


def test_oracle_quantise_rows_is_the_packer_s_rule():
    g = np.random.default_rng(2)
    from workload import f32_to_bf16_bits, bf16_bits_to_f32
    bits = f32_to_bf16_bits(g.standard_normal((9, 64)).astype(np.float32))
    packed, scales, t = oracle.quantize_ref(bf16_bits_to_f32(bits))
    codes, s = okv.quantise_rows(bits, t)
    assert np.array_equal(s, scales) and np.array_equal(codes[:, 0::2] | codes[:, 1::2] << 4, packed)


def test_oracle_attention_closed_forms():
    d = 64
    v = np.arange(10 * d, dtype=np.float64).reshape(10, d)
    k = np.zeros((10, d))
    out, lse, _, _ = okv.attention(np.ones((3, d)), k, v, 1.0)             # equal scores: means of what is seen
    for i, n in enumerate((8, 9, 10)):
        assert np.allclose(out[i], v[:n].mean(0)) and np.isclose(lse[i], np.log(n))
    out, _, _, _ = okv.attention(np.ones((3, d)), k, v, 1.0, window=2)
    for i, n in enumerate((8, 9, 10)):
        assert np.allclose(out[i], v[n - 2:n].mean(0))
    out, lse, _, _ = okv.attention(np.ones((3, d)), k[:1], v[:1], 1.0)     # two queries before the only slot
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.allclose(out[2], v[0])
    k[4, 0] = 1e3
    _, lse, _, _ = okv.attention(np.eye(1, d), k, v, 1.0, softcap=7.0)      # the cap bounds the score
    assert np.isclose(lse[0], np.log(9 + np.exp(7.0)))
    w, _ = okv.slot_weights(np.ones((2, d)), np.zeros((3, d)), np.log([2.0, 3.0]), 1.0)
    assert np.allclose(w, [1 / 2 + 1 / 3, 1 / 2 + 1 / 3, 1 / 3])


def test_oracle_evict_and_sample_closed_forms():
    w = np.array([0, 5, 1, 5, 2, 5, 0, 0], np.float32)
    assert okv.evict(w, 8, 4, 1, 1).tolist() == [0, 1, 3, 7]
    assert okv.evict(w, 3, 4, 1, 1).tolist() == [0, 1, 2]
    x = np.log(np.array([1, 2, 4, 1], np.float32)).astype(np.float32)
    for u, want in ((0.0, 0), (0.12, 0), (0.13, 1), (0.37, 1), (0.38, 2), (0.87, 2), (0.88, 3)):
        assert sample_ref(x, u)[0] == want
    assert sample_ref(x, 0.99, top_k=2)[0] == 2 and sample_ref(x, 0.1, top_k=2)[0] == 1
    assert sample_ref(x, 0.9, top_p=0.5)[0] == 2 and sample_ref(x, 0.3, temperature=0.0)[0] == 2
    assert sample_ref(x, 0.99, min_p=0.4)[0] == 2
    assert sample_ref(np.full(3, -np.inf, np.float32), 0.5)[0] == -1

"""The serving step around the NVFP4 products: a paged key/value cache held in
NVFP4 (append, read, attention, the weight each slot got, eviction) and the
choice of the next token.

Argument checks and marshalling only, as in the rest of the binding: every step
runs in the library's HIP kernels.  The C functions, the cache's layout and the
exact rules are in include/nvfp4_kv.h.  Calls run on `stream` (default: torch's
current stream of the tensors' device), never wait for the device, and write to
the tensors they return or were given; those must stay alive until the stream
has passed, as with any torch call on another stream.  Tensors and workspaces
that a call makes belong to `stream`, like what torch makes under
torch.cuda.stream(stream): to use a result elsewhere, wait for that stream, and
record_stream() the result if it is dropped while such work is under way.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _lib

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32   # a module's own names are found faster, which a one-token step notices
_empty, _raw_stream = torch.empty, torch._C._cuda_getCurrentRawStream

PAGE = 64
HEAD_DIMS = (64, 128, 256)
LOGITS_BF16, LOGITS_F32 = 0, 1

EXPORTED = ("nvfp4_kv_record_bytes", "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_kv_attention_workspace",
            "nvfp4_kv_attention", "nvfp4_kv_weights", "nvfp4_kv_evict", "nvfp4_sample", "nvfp4_sample_workspace")


class _Cache(ctypes.Structure):
    """nvfp4_kv_cache_t"""
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _Seqs(ctypes.Structure):
    """nvfp4_kv_seqs_t"""
    _fields_ = [("table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("table_pitch", ctypes.c_int64), ("seqs", ctypes.c_int64), ("total", ctypes.c_int64)]


class _Queries(ctypes.Structure):
    """nvfp4_kv_queries_t"""
    _fields_ = [("q", ctypes.c_void_p), ("q_pitch", ctypes.c_int64), ("q_head_pitch", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("max_q", ctypes.c_int64), ("max_kv", ctypes.c_int64),
                ("window", ctypes.c_int64), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("causal", ctypes.c_int32)]


_DECLARED = None


def _kv() -> ctypes.CDLL:
    global _DECLARED
    if _DECLARED is None:
        lib = _lib()
        vp, i64 = ctypes.c_void_p, ctypes.c_int64
        cache, seqs, queries = ctypes.POINTER(_Cache), ctypes.POINTER(_Seqs), ctypes.POINTER(_Queries)
        out = ctypes.POINTER(i64)
        lib.nvfp4_kv_record_bytes.argtypes = [i64, out]
        lib.nvfp4_kv_append.argtypes = [cache, seqs, vp, i64, i64, vp, i64, i64, vp]
        lib.nvfp4_kv_read.argtypes = [cache, seqs, vp, vp, vp]
        lib.nvfp4_kv_attention_workspace.argtypes = [cache, seqs, queries, out]
        lib.nvfp4_kv_attention.argtypes = [cache, seqs, queries, vp, vp, vp, i64, vp]
        lib.nvfp4_kv_weights.argtypes = [cache, seqs, queries, vp, vp, vp, vp]
        lib.nvfp4_kv_evict.argtypes = [cache, seqs, vp, i64, i64, i64, i64, cache, vp, i64, vp, vp, vp, vp]
        lib.nvfp4_sample.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]
        lib.nvfp4_sample_workspace.argtypes = [i64, i64, out]
        for name in EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        _DECLARED = lib
    return _DECLARED


class KvCache:
    """A paged NVFP4 key/value cache over `data`, uint8 [pages, kv_heads, 72 * head_dim].

    The tensor scales are fixed for the cache's life: a stored value is
    scale * e4m3 * e2m1, so values up to 2688 * scale are held."""

    def __init__(self, data, kv_heads: int, head_dim: int, k_scale: float, v_scale: float):
        if head_dim not in HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {HEAD_DIMS}")
        if data.dtype != torch.uint8 or data.dim() != 3 or tuple(data.shape[1:]) != (kv_heads, 72 * head_dim):
            raise ValueError(f"data must be uint8 [pages, {kv_heads}, {72 * head_dim}]")
        if not data.is_cuda or not data.is_contiguous():
            raise ValueError("data must be a contiguous GPU tensor")
        self.data, self.kv_heads, self.head_dim = data, int(kv_heads), int(head_dim)
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.pages, self.device = data.shape[0], data.device
        self._c = _Cache(data.data_ptr(), self.pages, self.kv_heads, self.head_dim, self.k_scale, self.v_scale)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, k_scale: float, v_scale: float, device="cuda") -> "KvCache":
        """A cache of `pages` pages of zeros."""
        data = torch.zeros((pages, kv_heads, 72 * head_dim), dtype=torch.uint8, device=device)
        return cls(data, kv_heads, head_dim, k_scale, v_scale)


def _ints(name, t, dim, device):
    if t.dtype is not _I32 or t.dim() != dim or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dim}-D int32 tensor on {device}")
    return t.data_ptr()


def _seqs(cache, table, kv_lens, q_starts, total) -> _Seqs:
    dev = cache.device
    seqs = kv_lens.shape[0]
    if table.shape[0] != seqs:
        raise ValueError("table and kv_lens must have one row and one length for each sequence")
    starts = 0
    if q_starts is not None:
        if q_starts.shape[0] != seqs + 1:
            raise ValueError("q_starts must hold one more entry than kv_lens")
        starts = _ints("q_starts", q_starts, 1, dev)
    return _Seqs(_ints("table", table, 2, dev), _ints("kv_lens", kv_lens, 1, dev), starts, table.shape[1], seqs, total)


def _rows(name, x, cache, heads=None):
    if x.dtype is not _BF16 or x.dim() != 3 or x.device != cache.device:
        raise ValueError(f"{name} must be a bf16 [tokens, heads, head_dim] tensor on {cache.device}")
    _, width, dim = x.shape
    pitch, head_pitch, step = x.stride()
    if dim != cache.head_dim or (heads is not None and width != heads) or step != 1:
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {cache.head_dim}] with contiguous rows")
    return x.data_ptr(), pitch, head_pitch


def _new(shape, dtype, device, stream):
    # from the pool of the stream that writes it: what another stream's pool hands out may still be in
    # use by work queued there
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return _empty(shape, dtype=dtype, device=device)


def _out(name, t, shape, dtype, device, stream=None):
    if t is None:
        return _new(shape, dtype, device, stream)
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _room(workspace, device):
    """Address and bytes of a workspace, or of none."""
    if workspace is None:
        return 0, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream(stream, device) -> int:
    # the raw handle at once: torch.cuda.current_stream() would build a Stream object (2 us) first
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def kv_append(cache: KvCache, k, v, table, kv_lens, q_starts, stream=None) -> None:
    """Quantises the new tokens' K and V rows (bf16 [total, kv_heads, head_dim], views with
    strides of multiples of 8 elements allowed) into each sequence's last slots."""
    seqs = _seqs(cache, table, kv_lens, q_starts, k.shape[0])
    if v.shape[0] != k.shape[0]:
        raise ValueError("k and v must hold the same tokens")
    _check(_kv().nvfp4_kv_append(cache._c, seqs, *_rows("k", k, cache, cache.kv_heads),
                                 *_rows("v", v, cache, cache.kv_heads), _stream(stream, cache.device)),
           "nvfp4_kv_append")


def kv_read(cache: KvCache, table, kv_lens, q_starts, total: int, k=None, v=None, stream=None):
    """The bf16 values of each sequence's last q_starts[s+1] - q_starts[s] slots: (k, v), each
    [total, kv_heads, head_dim]; rows without a slot are zeros."""
    shape = (total, cache.kv_heads, cache.head_dim)
    k = _out("k", k, shape, _BF16, cache.device, stream)
    v = _out("v", v, shape, _BF16, cache.device, stream)
    seqs = _seqs(cache, table, kv_lens, q_starts, total)
    _check(_kv().nvfp4_kv_read(cache._c, seqs, k.data_ptr(), v.data_ptr(), _stream(stream, cache.device)),
           "nvfp4_kv_read")
    return k, v


def _queries(cache, q, max_q, max_kv, scale, causal, window, softcap) -> _Queries:
    ptr, pitch, head_pitch = _rows("q", q, cache)
    return _Queries(ptr, pitch, head_pitch, q.shape[1], max_q, max_kv, window,
                    cache.head_dim ** -0.5 if scale is None else scale, softcap, 1 if causal else 0)


def kv_attention_workspace(cache: KvCache, q, table, kv_lens, q_starts, max_q: int, max_kv: int, window: int = 0) -> int:
    """Bytes of workspace that kv_attention takes for these arguments."""
    n = ctypes.c_int64()
    seqs = _seqs(cache, table, kv_lens, q_starts, q.shape[0])
    _check(_kv().nvfp4_kv_attention_workspace(cache._c, seqs, _queries(cache, q, max_q, max_kv, None, True, window, 0.0),
                                              n), "nvfp4_kv_attention_workspace")
    return n.value


def kv_attention(q, cache: KvCache, table, kv_lens, q_starts, max_q: int, max_kv: int, *, scale=None, causal=True,
                 window: int = 0, softcap: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens q (bf16 [total, heads, head_dim], strided views allowed) over the
    cache, their own slots included: (out bf16 [total, heads, head_dim], lse fp32 [total, heads]).

    max_q and max_kv bound every sequence's new tokens and length (host numbers, used to size the
    launch).  scale defaults to head_dim ** -0.5.  workspace: a uint8 tensor of
    kv_attention_workspace bytes (allocated when None; give one to capture a graph without torch's
    graph pools)."""
    dev = cache.device
    seqs = _seqs(cache, table, kv_lens, q_starts, q.shape[0])
    queries = _queries(cache, q, max_q, max_kv, scale, causal, window, softcap)
    out = _out("out", out, q.shape, _BF16, dev, stream)
    lse = _out("lse", lse, q.shape[:2], _F32, dev, stream)
    lib = _kv()
    if workspace is None:
        n = ctypes.c_int64()
        _check(lib.nvfp4_kv_attention_workspace(cache._c, seqs, queries, n), "nvfp4_kv_attention")
        if n.value:
            workspace = _new(n.value, torch.uint8, dev, stream)
    wp, wn = _room(workspace, dev)
    _check(lib.nvfp4_kv_attention(cache._c, seqs, queries, out.data_ptr(), lse.data_ptr(), wp, wn, _stream(stream, dev)),
           "nvfp4_kv_attention")
    return out, lse


def kv_weights(q, lse, cache: KvCache, table, kv_lens, q_starts, max_q: int, max_kv: int, *, scale=None, causal=True,
               window: int = 0, softcap: float = 0.0, prior=None, out=None, stream=None):
    """prior + the softmax weight each slot got from the new tokens q, summed over them and over the
    query heads of a kv head: fp32 [seqs, kv_heads, max_kv].  lse as kv_attention returned it for the
    same arguments; out may be prior (summed in place)."""
    dev = cache.device
    seqs = _seqs(cache, table, kv_lens, q_starts, q.shape[0])
    queries = _queries(cache, q, max_q, max_kv, scale, causal, window, softcap)
    shape = (seqs.seqs, cache.kv_heads, max_kv)
    out = _out("out", out, shape, _F32, dev, stream)
    if prior is not None:
        _out("prior", prior, shape, _F32, dev)
    _out("lse", lse, q.shape[:2], _F32, dev)
    _check(_kv().nvfp4_kv_weights(cache._c, seqs, queries, lse.data_ptr(), 0 if prior is None else prior.data_ptr(),
                                  out.data_ptr(), _stream(stream, dev)), "nvfp4_kv_weights")
    return out


def kv_evict(weights, cache: KvCache, table, kv_lens, dst_table, keep: int, *, sink: int = 0, recent: int = 0, dst=None,
             kept=None, kept_weights=None, new_lens=None, stream=None):
    """Cuts every sequence to at most `keep` slots a kv head: the first `sink`, the last `recent` and
    those between with the largest weights [seqs, kv_heads, n], copied in slot order into the pages
    of dst_table [seqs, at least keep / 64] of `dst` (default: the same cache; one with the same geometry
    and tensor scales, whose pages in dst_table no sequence of the call reads).  Returns (kept int32 [seqs, kv_heads, keep], their weights, the new
    lengths int32 [seqs])."""
    dev = cache.device
    dst = cache if dst is None else dst
    if dst.device != dev:
        raise ValueError(f"dst must be a cache on {dev}")
    seqs = _seqs(cache, table, kv_lens, None, 0)
    shape = (seqs.seqs, cache.kv_heads, keep)
    if weights.dim() != 3 or tuple(weights.shape[:2]) != shape[:2]:
        raise ValueError(f"weights must be [{shape[0]}, {shape[1]}, slots]")
    _out("weights", weights, weights.shape, _F32, dev)
    if dst_table.shape[0] != shape[0]:
        raise ValueError("dst_table must have one row for each sequence")
    dst_ptr = _ints("dst_table", dst_table, 2, dev)
    kept = _out("kept", kept, shape, _I32, dev, stream)
    kept_weights = _out("kept_weights", kept_weights, shape, _F32, dev, stream)
    new_lens = _out("new_lens", new_lens, shape[:1], _I32, dev, stream)
    _check(_kv().nvfp4_kv_evict(cache._c, seqs, weights.data_ptr(), weights.shape[2], keep, sink, recent, dst._c, dst_ptr,
                                dst_table.shape[1], kept.data_ptr(), kept_weights.data_ptr(), new_lens.data_ptr(),
                                _stream(stream, dev)), "nvfp4_kv_evict")
    return kept, kept_weights, new_lens


def _param(name, t, rows, dtype, device):
    if t is None:
        return 0
    return _out(name, t, (rows,), dtype, device).data_ptr()


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, *, token=None, logprob=None, workspace=None,
           stream=None):
    """One token a row of logits (bf16 or fp32 [rows, vocab], rows may be strided) from the row's
    random number u in [0, 1): (token int32 [rows], logprob fp32 [rows]).  temperature, top_p, min_p
    fp32 and top_k int32 are tensors [rows]; None stands for 1, 1, 0 and 0 (no limit)."""
    if logits.dtype not in (_BF16, _F32) or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a bf16 or float32 [rows, vocab] GPU tensor")
    if logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("logits must have contiguous rows")
    rows, vocab = logits.shape
    dev = logits.device
    f32 = logits.dtype is _F32
    token = _out("token", token, (rows,), _I32, dev, stream)
    logprob = _out("logprob", logprob, (rows,), _F32, dev, stream)
    lib = _kv()
    n = ctypes.c_int64()
    _check(lib.nvfp4_sample_workspace(rows, vocab, n), "nvfp4_sample")
    if workspace is None and n.value:
        workspace = _new(n.value, torch.uint8, dev, stream)
    wp, wn = _room(workspace, dev)
    _check(lib.nvfp4_sample(logits.data_ptr(), LOGITS_F32 if f32 else LOGITS_BF16, rows, vocab,
                            logits.stride(0) if rows > 1 else vocab, _param("u", u, rows, _F32, dev),
                            _param("temperature", temperature, rows, _F32, dev),
                            _param("top_k", top_k, rows, _I32, dev),
                            _param("top_p", top_p, rows, _F32, dev),
                            _param("min_p", min_p, rows, _F32, dev),
                            token.data_ptr(), logprob.data_ptr(), wp, wn, _stream(stream, dev)), "nvfp4_sample")
    return token, logprob

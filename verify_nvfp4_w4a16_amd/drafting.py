"""The verify round over drafted tokens, beside the cache and the sampler of
serving.py: the page tables of a step, what the nodes of a drafted tree see and
their attention, penalties, biases and grammar masks on logits, the branch that
the model accepts and its move in the cache.

Argument checks and marshalling only; every step runs in the library's HIP
kernels.  The C functions and the exact rules are in include/nvfp4_draft.h;
streams, workspaces and results are serving.py's.  Nothing waits for the device
and all lengths stay on it, so a round can be captured in one graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, _lib
from .serving import _BF16, _F32, _I32, LOGITS_BF16, LOGITS_F32, _Cache, _ints, _launch, _new, _out, _Queries, _queries, _room, _Seqs, _seqs

_I64 = torch.int64

TREE_MAX, TREE_WORDS, BIAS_MAX = 256, 4, 1024

EXPORTED = ("nvfp4_kv_pages", "nvfp4_kv_tree", "nvfp4_kv_tree_attention_workspace", "nvfp4_kv_tree_attention",
            "nvfp4_adjust_logits", "nvfp4_tree_accept", "nvfp4_kv_move")

_VP, _I = ctypes.c_void_p, ctypes.c_int64


class _Pages(ctypes.Structure):
    """nvfp4_kv_pages_t"""
    _fields_ = [("pool", _VP), ("state", _VP), ("capacity", _I), ("table", _VP), ("table_pitch", _I), ("held", _VP), ("keep", _VP),
                ("fresh", _VP), ("seqs", _I), ("total", _I)]


class _Tree(ctypes.Structure):
    """nvfp4_kv_tree_t"""
    _fields_ = [("masks", _VP), ("positions", _VP), ("words", _I), ("whole_tree", ctypes.c_int32)]


class _Adjust(ctypes.Structure):
    """nvfp4_adjust_t"""
    _fields_ = [("logits", _VP), ("rows", _I), ("vocab", _I), ("pitch", _I), ("out_pitch", _I), ("logits_type", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("q_starts", _VP), ("seqs", _I), ("history", _VP), ("history_lens", _VP),
                ("prompt_lens", _VP), ("history_pitch", _I), ("repetition", _VP), ("presence", _VP), ("frequency", _VP),
                ("bias_tokens", _VP), ("bias_values", _VP), ("bias_width", _I), ("allowed", _VP), ("allowed_rows", _VP),
                ("allowed_pitch", _I), ("states", _I), ("drafted", _VP), ("masks", _VP), ("mask_words", _I)]


_DECLARED = None


def _draft() -> ctypes.CDLL:
    global _DECLARED
    if _DECLARED is None:
        lib = _lib()
        cache, seqs, queries = ctypes.POINTER(_Cache), ctypes.POINTER(_Seqs), ctypes.POINTER(_Queries)
        lib.nvfp4_kv_pages.argtypes = [ctypes.POINTER(_Pages), _VP, _VP, _VP, _VP, _VP, _VP, _VP]
        lib.nvfp4_kv_tree.argtypes = [_VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP]
        lib.nvfp4_kv_tree_attention_workspace.argtypes = [cache, seqs, queries, ctypes.POINTER(_I)]
        lib.nvfp4_kv_tree_attention.argtypes = [cache, seqs, queries, ctypes.POINTER(_Tree), _VP, _VP, _VP, _I, _VP]
        lib.nvfp4_adjust_logits.argtypes = [ctypes.POINTER(_Adjust), _VP, _VP]
        lib.nvfp4_tree_accept.argtypes = [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _VP, _VP]
        lib.nvfp4_kv_move.argtypes = [cache, _I, seqs, _VP, _I, _VP]
        for name in EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        _DECLARED = lib
    return _DECLARED


def _gpu(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _array(name, t, shape, dtype, device):
    """Address of a contiguous tensor of this shape, type and device; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


class KvStep(NamedTuple):
    """The tables of a step (kv_pages); the page table itself is written in place."""
    state: torch.Tensor       # int32 [2]: the pool's head and count after the step
    held: torch.Tensor        # int32 [seqs]: pages each sequence owns after it
    kv_lens: torch.Tensor     # int32 [seqs]
    q_starts: torch.Tensor    # int32 [seqs + 1]
    slots: torch.Tensor       # int32 [total]: 64 * page + slot in page of each new token, -1 behind the last
    positions: torch.Tensor   # int32 [total]: its slot's number in the sequence, -1 behind the last


def kv_pages(pool, state, table, held, keep, fresh, total: int, *, out: KvStep = None, stream=None) -> KvStep:
    """The page table and the arrays of a step, made on the device from the slots that each sequence
    keeps and the new tokens that it asks for (int32 [seqs] both).

    pool (int32, at least as many entries as there are pages) is a ring of free page numbers: entry
    (head + i) % len(pool) for i < count, with state = [head, count].  table (int32 [seqs, pages])
    and held (int32 [seqs], entries of a row that the sequence owns) are the sequences' pages.  New
    pages come from the pool's front into table, pages that a sequence no longer needs go to its
    back, both in place; a sequence that ended keeps 0 slots and asks for none.  One whose pages or
    tokens (`total` rows at most) are not there keeps its slots and gets no new tokens.  The step's
    slots serve callers that write rows elsewhere themselves; kv_append takes the table.  out: the
    tensors to write; its state, held and kv_lens may be the call's own state, held and keep, so
    that a captured step carries them on."""
    dev = _gpu("table", table)
    seqs = held.shape[0]
    if table.dim() != 2 or table.shape[0] != seqs:
        raise ValueError("table must have one row for each entry of held")
    if total < 0:
        raise ValueError("total must be at least 0")
    p = _Pages(_ints("pool", pool, 1, dev), _array("state", state, (2,), _I32, dev), pool.shape[0], _ints("table", table, 2, dev),
               table.shape[1], _ints("held", held, 1, dev), _array("keep", keep, (seqs,), _I32, dev),
               _array("fresh", fresh, (seqs,), _I32, dev), seqs, total)
    if out is None:   # pieces of one tensor: an allocation costs the host more than a view
        out = KvStep(*_new(3 + 3 * seqs + 2 * total, _I32, dev, stream).split_with_sizes((2, seqs, seqs, seqs + 1, total, total)))
    else:
        for name, t, n in zip(KvStep._fields, out, (2, seqs, seqs, seqs + 1, total, total)):
            _array(name, t, (n,), _I32, dev)
    _launch("nvfp4_kv_pages", _draft().nvfp4_kv_pages, dev, stream, p, out.state.data_ptr(), out.held.data_ptr(),
            out.kv_lens.data_ptr(), out.q_starts.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr())
    return out


def _tree_seqs(kv_lens, q_starts, dev):
    seqs = kv_lens.shape[0]
    return _ints("kv_lens", kv_lens, 1, dev), _array("q_starts", q_starts, (seqs + 1,), _I32, dev), seqs


def kv_tree(parents, kv_lens, q_starts, max_q: int, *, masks=None, positions=None, stream=None):
    """What each node of the sequences' trees sees and where it stands: (masks int64 [total, ceil(max_q / 64)],
    bit a set for the ancestors a of a node and itself; positions int32 [total], the slots before the
    tree plus the node's depth).  parents int32 [total]: the node (counted within its tree, below
    its own place) that each continues, -1 for none; no tree has more than max_q nodes, 1..256."""
    dev = _gpu("parents", parents)
    lens, starts, seqs = _tree_seqs(kv_lens, q_starts, dev)
    up = _ints("parents", parents, 1, dev)
    total = parents.shape[0]
    if not 1 <= max_q <= TREE_MAX:
        raise ValueError(f"max_q must be 1..{TREE_MAX}")
    masks = _out("masks", masks, (total, (max_q + 63) // 64), _I64, dev, stream)
    positions = _out("positions", positions, (total,), _I32, dev, stream)
    _launch("nvfp4_kv_tree", _draft().nvfp4_kv_tree, dev, stream, up, lens, starts, seqs, total, max_q, masks.data_ptr(),
            positions.data_ptr())
    return masks, positions


def kv_tree_attention_workspace(cache, q, table, kv_lens, q_starts, max_q: int, max_kv: int, window: int = 0) -> int:
    """Bytes of workspace that kv_tree_attention takes for these arguments."""
    n = _I()
    _check(_draft().nvfp4_kv_tree_attention_workspace(cache._c, _seqs(cache, table, kv_lens, q_starts, q.shape[0]),
                                                      _queries(cache, q, max_q, max_kv, None, True, window, 0.0), n),
           "nvfp4_kv_tree_attention_workspace")
    return n.value


def kv_tree_attention(q, cache, table, kv_lens, q_starts, masks, positions, max_q: int, max_kv: int, *, scale=None,
                      window: int = 0, softcap: float = 0.0, whole_tree: bool = False, out=None, lse=None, workspace=None, stream=None):
    """kv_attention for the nodes of trees: each row of q (bf16 [total, heads, head_dim]) sees the
    slots before its tree and, of the tree's own, the ones its mask names; with a window, of both those
    at positions after its own - window.  masks int64 [total, words] and positions int32 [total] as
    kv_tree gives them; positions may be None where there is no window.  whole_tree: the window counts
    before the tree alone, for masks that say all about the tree itself.  No tree has more than max_q
    nodes (at most 256).  The rest is kv_attention's.

    max_q and max_kv also choose the kernel: a capacity as the bound, as a captured round takes it, costs
    short caches up to three times the time."""
    dev = cache.device
    total = q.shape[0]
    seqs = _seqs(cache, table, kv_lens, q_starts, total)
    queries = _queries(cache, q, max_q, max_kv, scale, True, window, softcap)
    if masks.dim() != 2:
        raise ValueError("masks must be int64 [total, words]")
    tree = _Tree(_array("masks", masks, (total, masks.shape[1]), _I64, dev), _array("positions", positions, (total,), _I32, dev),
                 masks.shape[1], bool(whole_tree))
    out = _out("out", out, q.shape, _BF16, dev, stream)
    lse = _out("lse", lse, q.shape[:2], _F32, dev, stream)
    lib = _draft()
    if workspace is None:
        n = _I()
        _check(lib.nvfp4_kv_tree_attention_workspace(cache._c, seqs, queries, n), "nvfp4_kv_tree_attention")
        if n.value:
            workspace = _new(n.value, torch.uint8, dev, stream)
    wp, wn = _room(workspace, dev)
    _launch("nvfp4_kv_tree_attention", lib.nvfp4_kv_tree_attention, dev, stream, cache._c, seqs, queries, tree, out.data_ptr(),
            lse.data_ptr(), wp, wn)
    return out, lse


def _logits(name, t):
    if t.dtype not in (_BF16, _F32) or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a bf16 or float32 [rows, vocab] GPU tensor")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1], LOGITS_F32 if t.dtype is _F32 else LOGITS_BF16


def adjust_logits(logits, history=None, history_lens=None, *, prompt_lens=None, q_starts=None, repetition=None, presence=None,
                  frequency=None, bias_tokens=None, bias_values=None, allowed=None, allowed_rows=None, drafted=None, masks=None,
                  out=None, stream=None):
    """Logits [rows, vocab] (bf16 or fp32, rows may be strided) with the penalties of what was said,
    biases and grammar masks, in a new tensor of their type or in `out` (of either type; may be logits
    itself).

    Rows q_starts[s] .. q_starts[s + 1] - 1 are sequence s's; without q_starts row r is sequence r.
    history int32 [seqs, n]: the sequence's tokens, history_lens [seqs] of them, the first prompt_lens
    [seqs] its prompt.  With n the times a token stands in it after the prompt:
      repetition  fp32 [seqs]: x / r where x > 0, else x * r, for tokens of the prompt or with n > 0
      presence, frequency  fp32 [seqs]: x - p - f n for tokens with n > 0
      bias_tokens int32, bias_values fp32 [seqs, up to 1024]: added (a negative token is none; the last of equal ones counts)
      allowed     int32 [states, ceil(vocab / 32)]: bit v % 32 of word v / 32 says that token v may come; the others
                  become -inf.  allowed_rows int32 [rows] is each row's state, a negative one none (default: state r).
    drafted int32 [rows] and masks int64 [rows, words] (kv_tree's) count the tokens on a node's way too."""
    pitch, kind = _logits("logits", logits)
    rows, vocab = logits.shape
    dev = logits.device
    seqs = rows if q_starts is None else q_starts.shape[0] - 1
    if q_starts is not None:
        starts = _ints("q_starts", q_starts, 1, dev)
        if seqs < 0:
            raise ValueError("q_starts must hold one more entry than there are sequences")
    else:
        starts = 0
    if history is None and (history_lens is not None or prompt_lens is not None):
        raise ValueError("history_lens and prompt_lens go with history")
    width = 0
    if history is not None:
        if history_lens is None or history.dim() != 2:
            raise ValueError("history must be int32 [seqs, n] with history_lens")
        width = history.shape[1]
    if (bias_tokens is None) != (bias_values is None) or (drafted is None) != (masks is None):
        raise ValueError("bias_tokens go with bias_values, and drafted with masks")
    if allowed is None and allowed_rows is not None:
        raise ValueError("allowed_rows go with allowed")
    for name, t in (("bias_tokens", bias_tokens), ("allowed", allowed), ("masks", masks)):
        if t is not None and t.dim() != 2:
            raise ValueError(f"{name} must have two dimensions")
    if out is None:
        out = _new((rows, vocab), logits.dtype, dev, stream)
        out_pitch, out_kind = vocab, kind
    else:
        out_pitch, out_kind = _logits("out", out)
        if out.shape != logits.shape or out.device != dev:
            raise ValueError(f"out must be [{rows}, {vocab}] on {dev}")
    a = _Adjust(logits.data_ptr(), rows, vocab, pitch, out_pitch, kind, out_kind, starts, seqs,
                _array("history", history, (seqs, width), _I32, dev), _array("history_lens", history_lens, (seqs,), _I32, dev),
                _array("prompt_lens", prompt_lens, (seqs,), _I32, dev), width,
                _array("repetition", repetition, (seqs,), _F32, dev), _array("presence", presence, (seqs,), _F32, dev),
                _array("frequency", frequency, (seqs,), _F32, dev))
    if bias_tokens is not None:
        a.bias_width = bias_tokens.shape[1]
        a.bias_tokens = _array("bias_tokens", bias_tokens, (seqs, a.bias_width), _I32, dev)
        a.bias_values = _array("bias_values", bias_values, (seqs, a.bias_width), _F32, dev)
    if allowed is not None:
        a.states, a.allowed_pitch = allowed.shape
        if a.allowed_pitch * 32 < vocab:   # an empty tensor has no address to tell the library that it was given
            raise ValueError(f"allowed must hold a bit for each of {vocab} tokens")
        a.allowed = _array("allowed", allowed, allowed.shape, _I32, dev)
        a.allowed_rows = _array("allowed_rows", allowed_rows, (rows,), _I32, dev)
    if drafted is not None:
        a.mask_words = masks.shape[1]
        a.drafted = _array("drafted", drafted, (rows,), _I32, dev)
        a.masks = _array("masks", masks, (rows, a.mask_words), _I64, dev)
    _launch("nvfp4_adjust_logits", _draft().nvfp4_adjust_logits, dev, stream, a, out.data_ptr())
    return out


def tree_accept(drafted, parents, chosen, kv_lens, q_starts, max_q: int, *, path=None, counts=None, token=None, new_lens=None,
                stream=None):
    """The branch of each tree that the model goes along: from node 0 on to the continuation whose
    drafted token is the one chosen at the node (int32 [total] all three, `chosen` as sample gives it
    for the nodes' logits).  Returns (path int32 [seqs, max_q], the nodes taken and then -1; counts
    [seqs]; token [seqs], what is chosen after the last of them; new_lens [seqs], the slots that stay)."""
    dev = _gpu("parents", parents)
    lens, starts, seqs = _tree_seqs(kv_lens, q_starts, dev)
    total = parents.shape[0]
    if not 1 <= max_q <= TREE_MAX:
        raise ValueError(f"max_q must be 1..{TREE_MAX}")
    if path is counts is token is new_lens is None:   # pieces of one tensor, as kv_pages has them
        path, counts, token, new_lens = _new(seqs * (max_q + 3), _I32, dev, stream).split_with_sizes((seqs * max_q, seqs, seqs, seqs))
        path = path.view(seqs, max_q)
    else:
        path = _out("path", path, (seqs, max_q), _I32, dev, stream)
        counts = _out("counts", counts, (seqs,), _I32, dev, stream)
        token = _out("token", token, (seqs,), _I32, dev, stream)
        new_lens = _out("new_lens", new_lens, (seqs,), _I32, dev, stream)
    _launch("nvfp4_tree_accept", _draft().nvfp4_tree_accept, dev, stream, _array("drafted", drafted, (total,), _I32, dev),
            _ints("parents", parents, 1, dev), _array("chosen", chosen, (total,), _I32, dev), lens, starts, seqs, total, max_q,
            path.data_ptr(), counts.data_ptr(), token.data_ptr(), new_lens.data_ptr())
    return path, counts, token, new_lens


def kv_move(caches, table, kv_lens, q_starts, path, *, stream=None) -> None:
    """Moves the slots of each sequence's path (int32 [seqs, max_q], tree_accept's) to the front of its
    tree, in one cache or in every one of a list (the layers of a model: one geometry, one table, no
    data in common).  kv_lens and q_starts are the tree's; afterwards tree_accept's new_lens hold."""
    caches = (caches,) if hasattr(caches, "_c") else tuple(caches)
    if not caches:
        raise ValueError("caches must hold at least one cache")
    first = caches[0]
    if any(c.device != first.device for c in caches):
        raise ValueError(f"all caches must be on {first.device}")
    if path.dim() != 2:
        raise ValueError("path must be int32 [seqs, max_q]")
    max_q = path.shape[1]
    # no packed tensor is touched, so starts are held to nothing but what any call can have
    seqs = _seqs(first, table, kv_lens, q_starts, 1 << 24)
    _launch("nvfp4_kv_move", _draft().nvfp4_kv_move, first.device, stream, (_Cache * len(caches))(*(c._c for c in caches)),
            len(caches), seqs, _array("path", path, (seqs.seqs, max_q), _I32, first.device), max_q)

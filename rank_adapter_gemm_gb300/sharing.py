"""Binding of include/lora_sharing.h: requests that share what they have cached.

Beams and parallel samples of one step: ``BeamSelect.run`` picks the continuations,
``PageTables.fork`` makes the next batch's block table from their parents,
``KVLayers.copy`` copies the pages that two rows would else write to, and, after
the step's ``KVStep.build`` and ``Rope.append``, ``SharedAttention.run`` attends with
each group's common prefix read once.  ``PageTables.compact`` moves the pages in
use to the front of the cache.  As in the rest of the binding, the ``lora_*``
functions carry the C names and pass addresses, strides and the current stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import _dev, _torch
from . import attention as _att
from ._lib import (LOGITS_TYPES, LORA_MAX_KV_LAYERS, LORA_MAX_SEQS, SHARE_MODES, check, load, lora_attention_t, lora_kv_t,
                   lora_prefix_t)
from .attention import PagedKV, _flat, _matrix, _on, _table


def _ready():
    if _att._C is None:
        _att._types()
    return _att


def _opt(t, name, dtype, n=None) -> Optional[int]:
    return None if t is None else _flat(t, name, dtype, n)


def _rows(t, n):
    """(address, row stride, width) of a block table; the strides of one without rows mean nothing."""
    if n == 0 and getattr(t, "dtype", None) is _att._I32 and t.is_cuda and t.dim() == 2 and t.shape[0] == 0:
        return t.data_ptr(), t.shape[1], t.shape[1]
    return _table(t, n)


def _jobs(t, name, rows=None):
    """(address, rows) of an int32 [rows, 3] list of copies."""
    a = _flat(t, name, _att._I32)
    if t.dim() != 2 or t.shape[1] != 3 or (rows is not None and t.shape[0] < rows):
        raise ValueError(f"{name} must be an int32 [n, 3] tensor" + (f" of at least {rows} rows" if rows else ""))
    return a, t.shape[0]


def lora_beam_select_workspace_bytes(n_req: int, beams: int, keep: int, vocab: int) -> int:
    out = ctypes.c_size_t(0)
    check(load().lora_beam_select_workspace_bytes(int(n_req), int(beams), int(keep), int(vocab), ctypes.byref(out)),
          "lora_beam_select_workspace_bytes")
    return int(out.value)


def lora_beam_select(logits, scores, ended, beams: int, keep: int, eos: int, parents, tokens, out_scores, out_ended,
                     ws, stream=None) -> None:
    """logits: bf16 or fp32 [n_req * beams, vocab]; ended may be None."""
    T = _ready()
    _dev(logits, "logits")
    if logits.dtype is not T._BF16 and logits.dtype is not T._F32:
        raise TypeError("logits must be bf16 or fp32")
    kind = LOGITS_TYPES["bf16" if logits.dtype is T._BF16 else "fp32"]
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a 2-D tensor with unit column stride")
    rows, vocab = logits.shape
    if beams < 1 or rows % beams != 0:
        raise ValueError("logits must have a whole number of requests' beams")
    n = rows // beams
    ld = logits.stride(0) if rows > 1 else max(vocab, 1)
    if not (ws.is_cuda and ws.is_contiguous()):
        _dev(ws, "ws")
        raise ValueError("ws must be contiguous")
    status = load().lora_beam_select(
        logits.data_ptr(), ld, kind, n, beams, vocab, keep, _flat(scores, "scores", T._F32, rows),
        _opt(ended, "ended", T._I32, rows), eos, _flat(parents, "parents", T._I32, n * keep),
        _flat(tokens, "tokens", T._I32, n * keep), _flat(out_scores, "out_scores", T._F32, n * keep),
        _flat(out_ended, "out_ended", T._I32, n * keep), ws.data_ptr(), ws.numel() * ws.element_size(), _on(stream))
    if status:
        check(status, "lora_beam_select")


def lora_kv_fork(src_table, src_lens, parents, page_size: int, dst_table, dst_lens, copies, free_pages, n_free, err,
                 held=None, stream=None) -> None:
    """The cache's number of pages is free_pages.numel()."""
    T = _ready()
    n_src, n_dst = src_lens.numel(), parents.numel()
    src, ld_src, src_width = _rows(src_table, n_src)
    dst, ld_dst, dst_width = _rows(dst_table, n_dst)
    status = load().lora_kv_fork(
        src, ld_src, src_width, _flat(src_lens, "src_lens", T._I32), n_src, _flat(parents, "parents", T._I32), n_dst,
        page_size, free_pages.numel(), _opt(held, "held", T._I32), 0 if held is None else held.numel(), dst, ld_dst,
        dst_width, _flat(dst_lens, "dst_lens", T._I32, n_dst), _jobs(copies, "copies", n_dst)[0],
        _flat(free_pages, "free_pages", T._I32), _flat(n_free, "n_free", T._I32, 1), _opt(err, "err", T._I32),
        _on(stream))
    if status:
        check(status, "lora_kv_fork")


def lora_kv_compact(src_table, lens, page_size: int, dst_table, moves, n_moves, free_pages, n_free, err, held=None,
                    new_held=None, stream=None) -> None:
    """The cache's number of pages is free_pages.numel()."""
    T = _ready()
    n = lens.numel()
    src, ld_src, width = _rows(src_table, n)
    dst, ld_dst, dst_width = _rows(dst_table, n)
    if dst_width != width:
        raise ValueError("the tables must have the same width")
    n_held = 0 if held is None else held.numel()
    if n_held and new_held is None:
        raise ValueError("held pages need new_held")
    pages = free_pages.numel()
    status = load().lora_kv_compact(
        src, ld_src, width, _flat(lens, "lens", T._I32), n, page_size, pages, _opt(held, "held", T._I32), n_held, dst,
        ld_dst, _opt(new_held, "new_held", T._I32, n_held), _jobs(moves, "moves", pages // 2)[0],
        _flat(n_moves, "n_moves", T._I32, 1), _flat(free_pages, "free_pages", T._I32),
        _flat(n_free, "n_free", T._I32, 1), _opt(err, "err", T._I32), _on(stream))
    if status:
        check(status, "lora_kv_compact")


def lora_kv_copy(kvs, n_layers: int, copies, err, count=None, stream=None) -> None:
    """kvs: a ctypes array of lora_kv_t (KVLayers.c)."""
    T = _ready()
    at, n = _jobs(copies, "copies")
    status = load().lora_kv_copy(kvs, n_layers, at, n, _opt(count, "count", T._I32, 1), _opt(err, "err", T._I32),
                                 _on(stream))
    if status:
        check(status, "lora_kv_copy")


def lora_attend_shared_workspace_bytes(att: lora_attention_t, kv: lora_kv_t, T: int, n_seq: int) -> int:
    out = ctypes.c_size_t(0)
    check(load().lora_attend_shared_workspace_bytes(att, kv, int(T), int(n_seq), ctypes.byref(out)),
          "lora_attend_shared_workspace_bytes")
    return int(out.value)


def lora_attend_shared(q, out, q_offsets, kv_lens, block_table, group_offsets, prefix_lens, kv: lora_kv_t,
                       att: lora_attention_t, ws, err, max_q_hint: int = 0, lse=None, share: str = "auto",
                       stream=None) -> None:
    A = _ready()
    n, groups = kv_lens.numel(), prefix_lens.numel()
    x, ldq, T, q_cols = _matrix(q, "q")
    o, ldo, rows, o_cols = _matrix(out, "out")
    cols = att.n_heads * kv.head_dim
    if rows != T or q_cols < cols or o_cols < cols:
        raise ValueError("q and out must have the same rows and n_heads * head_dim columns")
    table, ld, width = _table(block_table, n)
    if not (ws.is_cuda and ws.is_contiguous()):
        _dev(ws, "ws")
        raise ValueError("ws must be contiguous")
    prefix = lora_prefix_t(_flat(group_offsets, "group_offsets", A._I32, groups + 1),
                           _flat(prefix_lens, "prefix_lens", A._I32), groups, SHARE_MODES[share])
    status = load().lora_attend_shared(
        x, ldq, o, ldo, _opt(lse, "lse", A._F32, T * att.n_heads), T, n, _flat(q_offsets, "q_offsets", A._I32, n + 1),
        _flat(kv_lens, "kv_lens", A._I32), table, ld, width, prefix, kv, att, max_q_hint, ws.data_ptr(),
        ws.numel() * ws.element_size(), _opt(err, "err", A._I32), _on(stream))
    if status:
        check(status, "lora_attend_shared")


class BeamSelect:
    """Selection of the `keep` best continuations of each of n_req requests with
    `beams` beams: its outputs (parents, tokens, scores, ended: flat, `keep` a
    request) and workspace.  Where keep = beams, ``scores`` and ``ended`` may be passed to
    the next call as they are."""

    def __init__(self, n_req: int, beams: int, keep: int, vocab: int, eos: int = -1, dtype=None, device="cuda"):
        torch = _torch()
        if dtype not in (None, torch.bfloat16, torch.float32):
            raise TypeError("logits are bf16 or fp32")
        self.n_req, self.beams, self.keep, self.vocab, self.eos = int(n_req), int(beams), int(keep), int(vocab), int(eos)
        self.dtype = dtype or torch.bfloat16
        size = lora_beam_select_workspace_bytes(n_req, beams, keep, vocab)
        self.ws = torch.zeros(size, dtype=torch.uint8, device=device)
        n = self.n_req * self.keep
        self.parents, self.tokens, self.ended = (torch.zeros(n, dtype=torch.int32, device=device) for _ in range(3))
        self.scores = torch.zeros(n, dtype=torch.float32, device=device)

    def run(self, logits, scores, ended=None, stream=None) -> None:
        if logits.dtype != self.dtype or tuple(logits.shape) != (self.n_req * self.beams, self.vocab):
            raise ValueError(f"logits must be {self.dtype} [{self.n_req * self.beams}, {self.vocab}]")
        if self.keep != self.beams and (scores is self.scores or (ended is not None and ended is self.ended)):
            raise ValueError("only where keep = beams may the last call's scores and ended be the next one's inputs")
        lora_beam_select(logits, scores, ended, self.beams, self.keep, self.eos, self.parents, self.tokens,
                         self.scores, self.ended, self.ws, stream)


class KVLayers:
    """The caches of a model's layers, of one geometry, for copies of pages in all of them."""

    def __init__(self, kvs: Sequence[PagedKV]):
        if not 1 <= len(kvs) <= LORA_MAX_KV_LAYERS:
            raise ValueError(f"between 1 and {LORA_MAX_KV_LAYERS} layers")
        self.kvs = list(kvs)
        self.c = (lora_kv_t * len(kvs))(*(kv.c for kv in kvs))

    def copy(self, copies, err, count=None, stream=None) -> None:
        """Page copies (rows of source, destination, tokens) in every layer."""
        lora_kv_copy(self.c, len(self.kvs), copies, err, count, stream)


class PageTables:
    """A batch's block table and lengths, and the free pages of its cache, over forks
    and compactions.  ``block_table`` (for KVStep and the attention) and ``lens`` are the
    current batch's; ``free_pages`` lists the free ids (then -1), ``copies`` the page copies
    that the last call asks for (``KVLayers.copy(tables.copies, tables.err, tables.n_copies)``).
    Rows change with fork; there is room for n_seq of them, and len(lens) in use."""

    def __init__(self, n_seq: int, max_pages: int, page_size: int, n_pages: int, device="cuda"):
        torch = _torch()
        if not 0 <= n_seq <= LORA_MAX_SEQS:
            raise ValueError(f"between 0 and {LORA_MAX_SEQS} requests")
        i32 = dict(dtype=torch.int32, device=device)
        self.n_seq, self.page_size, self.n_pages = int(n_seq), int(page_size), int(n_pages)
        self._tables = [torch.zeros(n_seq, max_pages, **i32) for _ in range(2)]
        self._lens = [torch.zeros(n_seq, **i32) for _ in range(2)]
        self._now, self._at, self._rows = 0, 0, self.n_seq  # table, lengths, rows
        self._fork_copies = torch.full((n_seq, 3), -1, **i32)
        self._moves = torch.full((n_pages // 2, 3), -1, **i32)
        self._n_moves = torch.zeros(1, **i32)
        self.copies, self.n_copies = self._fork_copies[:0], None
        self.free_pages = torch.arange(n_pages, **i32)
        self.n_free = torch.full((1,), n_pages, **i32)
        self.err = torch.zeros(1, **i32)

    @property
    def block_table(self):
        return self._tables[self._now][:self._rows]

    @property
    def lens(self):
        return self._lens[self._at][:self._rows]

    def fork(self, parents, held=None, stream=None) -> None:
        """Row i of the batch from here on continues row parents[i] (-1: empty)."""
        n, new, at = parents.numel(), 1 - self._now, 1 - self._at
        if n > self.n_seq:
            raise ValueError(f"room for {self.n_seq} requests")
        copies = self._fork_copies[:n]
        lora_kv_fork(self.block_table, self.lens, parents, self.page_size, self._tables[new][:n], self._lens[at][:n],
                     copies, self.free_pages, self.n_free, self.err, held, stream)
        self._now, self._at, self._rows, self.copies, self.n_copies = new, at, n, copies, None

    def compact(self, held=None, new_held=None, stream=None) -> None:
        """Pages in use to the front of the cache; new_held gets the held pages' new ids."""
        new = 1 - self._now
        lora_kv_compact(self.block_table, self.lens, self.page_size, self._tables[new][:self._rows], self._moves,
                        self._n_moves, self.free_pages, self.n_free, self.err, held, new_held, stream)
        self._now, self.copies, self.n_copies = new, self._moves, self._n_moves


class SharedAttention:
    """One layer's attention for a batch whose groups of requests share prefixes: room
    for T rows of n_seq requests; its parameters, workspace and error word.  Layers whose
    calls do not overlap can share one by passing ``kv``."""

    def __init__(self, n_seq: int, T: int, n_heads: int, kv: PagedKV, scale: Optional[float] = None,
                 softcap: float = 0.0, window: int = 0, slopes=None, device="cuda"):
        torch = _torch()
        if not 0 <= n_seq <= LORA_MAX_SEQS:
            raise ValueError(f"between 0 and {LORA_MAX_SEQS} requests")
        self.n_seq, self.T, self.kv, self.slopes = int(n_seq), int(T), kv, slopes
        if slopes is not None:
            _flat(slopes, "slopes", torch.float32, int(n_heads))
        scale = float(kv.c.head_dim) ** -0.5 if scale is None else float(scale)
        self.c = lora_attention_t(int(n_heads), scale, float(softcap or 0.0), int(window or 0),
                                  slopes.data_ptr() if slopes is not None else None)
        self.ws = torch.zeros(lora_attend_shared_workspace_bytes(self.c, kv.c, T, n_seq), dtype=torch.uint8,
                              device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def run(self, q, out, q_offsets, kv_lens, block_table, group_offsets, prefix_lens, max_q_hint: int = 0,
            kv: Optional[PagedKV] = None, lse=None, share: str = "auto", stream=None) -> None:
        """out = attention of q's rows; requests group_offsets[g] .. group_offsets[g + 1] - 1 hold the same keys and
        values below prefix_lens[g]; max_q_hint is an upper bound on a request's rows (0: taken as T / n_seq).
        share: "auto" reads prefixes once where that saves time, "always" all of them."""
        lora_attend_shared(q, out, q_offsets, kv_lens, block_table, group_offsets, prefix_lens, (kv or self.kv).c,
                           self.c, self.ws, self.err, max_q_hint, lse, share, stream)

"""Binding of include/lora_attention.h: the attention side of a serving step.

Per step ``KVStep.build`` writes the block tables, slot map and positions from
the requests' lengths; per layer ``Rope.append`` turns q and k of the packed
projection and writes k and v into the layer's ``PagedKV``, and
``Attention.run`` attends over it.  As in the rest of the binding, the
``lora_*`` functions carry the C names and pass addresses, strides and the
current stream; the classes only hold the caller-owned buffers.
"""
from __future__ import annotations

import ctypes
from typing import Mapping, Optional

import numpy as np

from . import _dev, _p, _torch
from ._lib import (ATTEND_PATHS, LORA_MAX_SEQS, ROPE_KINDS, check, load, lora_attention_t, lora_kv_t,
                   lora_rope_scaling_t, lora_rope_t)


# The checks below run on every call of a decode loop: they read each property
# once and leave the wording of a refusal to the slow path.  torch is loaded with
# the first call, as in the rest of the binding.
_I32 = _I64 = _F32 = _BF16 = _C = None


def _types():
    global _I32, _I64, _F32, _BF16, _C
    torch = _torch()
    _I32, _I64, _F32, _BF16, _C = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch._C


def _flat(t, name, dtype, n=None) -> int:
    """Address of a contiguous device tensor of n elements (any number: None)."""
    if getattr(t, "dtype", None) is dtype and t.is_cuda and t.is_contiguous() and (n is None or t.numel() == n):
        return t.data_ptr()
    _dev(t, name, dtype)
    raise ValueError(f"{name} must be contiguous" + (f" with {n} elements" if n is not None else ""))


def _table(t, n_seq):
    """(address, row stride, width) of a block table."""
    if getattr(t, "dtype", None) is _I32 and t.is_cuda and t.dim() == 2:
        rows, width = t.shape
        ld, one = t.stride()
        if rows == n_seq and (one == 1 or width <= 1):
            if ld >= width:
                return t.data_ptr(), ld, width
            if rows <= 1:  # the stride of a single row means nothing
                return t.data_ptr(), width, width
    _dev(t, "block_table", _I32)
    raise ValueError("block_table must be a 2-D int32 tensor, one row a request, with unit column stride and rows "
                     "that do not overlap")


def _matrix(t, name):
    """(address, row stride, rows, columns) of bf16 rows."""
    if getattr(t, "dtype", None) is _BF16 and t.is_cuda and t.dim() == 2:
        rows, cols = t.shape
        ld, one = t.stride()
        if one == 1:
            return t.data_ptr(), ld, rows, cols
    _dev(t, name, _BF16)
    raise ValueError(f"{name} must be a 2-D bf16 tensor with unit column stride")


def _on(stream) -> int:
    """A stream's address; the current one's without building a Stream object (2.8 us on a Grace core)."""
    return _C._cuda_getCurrentRawStream(_C._cuda_getDevice()) if stream is None else stream.cuda_stream


def lora_kv_step(ctx_lens, new_lens, page_size, free_pages, block_table, q_offsets, kv_lens, positions, seq_ids,
                 slot_map, taken, err, stream=None) -> None:
    if _C is None:
        _types()
    n, T = ctx_lens.numel(), positions.numel()
    table, ld, width = _table(block_table, n)
    status = load().lora_kv_step(
        _flat(ctx_lens, "ctx_lens", _I32), _flat(new_lens, "new_lens", _I32, n), n, page_size,
        _flat(free_pages, "free_pages", _I32), free_pages.numel(), table, ld, width, T,
        _flat(q_offsets, "q_offsets", _I32, n + 1), _flat(kv_lens, "kv_lens", _I32, n),
        _flat(positions, "positions", _I32), _flat(seq_ids, "seq_ids", _I32, T), _flat(slot_map, "slot_map", _I64, T),
        _flat(taken, "taken", _I32, 1), None if err is None else _flat(err, "err", _I32), _on(stream))
    if status:
        check(status, "lora_kv_step")


def lora_rope_phases(rot_dim: int, theta: float, scaling: Optional[Mapping] = None):
    """(uint64 phases [rot_dim / 2], factor on cos and sin) of a model's rotary
    frequencies; scaling: {"kind": "linear" | "ntk" | "llama3" | "yarn", "factor": ...}
    and, by kind, low_freq_factor, high_freq_factor, beta_fast, beta_slow, original."""
    sc = None
    if scaling is not None:
        fields = dict(scaling)
        kind = fields.pop("kind")
        if kind not in ROPE_KINDS:
            raise ValueError(f"unknown rotary scaling {kind!r}")
        known = {name for name, _ in lora_rope_scaling_t._fields_}
        if not set(fields) <= known:
            raise ValueError(f"unknown rotary scaling fields {sorted(set(fields) - known)}")
        sc = lora_rope_scaling_t(kind=ROPE_KINDS[kind], **{k: float(v) for k, v in fields.items()})
    phases = np.zeros(max(int(rot_dim) // 2, 1), np.uint64)
    mscale = ctypes.c_float(0.0)
    check(load().lora_rope_phases(int(rot_dim), float(theta), ctypes.byref(sc) if sc is not None else None,
                                  _p(phases), ctypes.byref(mscale)), "lora_rope_phases")
    return phases, float(mscale.value)


def lora_rope_append(qkv, q_out, n_heads, rope: lora_rope_t, positions, slot_map, kv: lora_kv_t, err,
                     stream=None) -> None:
    if _C is None:
        _types()
    x, ldx, T, cols = _matrix(qkv, "qkv")
    q, ldq, rows, q_cols = _matrix(q_out, "q_out")
    hd = kv.head_dim
    if rows != T or cols != (n_heads + 2 * kv.n_kv) * hd or q_cols < n_heads * hd:
        raise ValueError("qkv must have n_heads + 2 n_kv heads and q_out n_heads heads, with the same rows")
    status = load().lora_rope_append(
        x, ldx, T, n_heads, rope, _flat(positions, "positions", _I32, T), _flat(slot_map, "slot_map", _I64, T), q, ldq,
        kv, None if err is None else _flat(err, "err", _I32), _on(stream))
    if status:
        check(status, "lora_rope_append")


def lora_attend_workspace_bytes(att: lora_attention_t, kv: lora_kv_t) -> int:
    out = ctypes.c_size_t(0)
    check(load().lora_attend_workspace_bytes(att, kv, ctypes.byref(out)), "lora_attend_workspace_bytes")
    return int(out.value)


def lora_attend_resolve_path(path: str, att: lora_attention_t, kv: lora_kv_t, n_seq: int, max_q_hint: int) -> str:
    """The path lora_attend takes for n_seq requests of at most max_q_hint rows."""
    code = load().lora_attend_resolve_path(ATTEND_PATHS[path], att, kv, int(n_seq), int(max_q_hint))
    return {v: k for k, v in ATTEND_PATHS.items()}[int(code)]


def lora_attend(q, out, q_offsets, kv_lens, block_table, kv: lora_kv_t, att: lora_attention_t, ws, err,
                max_q_hint: int = 0, lse=None, path: str = "auto", stream=None) -> None:
    if _C is None:
        _types()
    n = kv_lens.numel()
    x, ldq, T, q_cols = _matrix(q, "q")
    o, ldo, rows, o_cols = _matrix(out, "out")
    cols = att.n_heads * kv.head_dim
    if rows != T or q_cols < cols or o_cols < cols:
        raise ValueError("q and out must have the same rows and n_heads * head_dim columns")
    table, ld, width = _table(block_table, n)
    if not (ws.is_cuda and ws.is_contiguous()):
        _dev(ws, "ws")
        raise ValueError("ws must be contiguous")
    status = load().lora_attend(
        x, ldq, o, ldo, None if lse is None else _flat(lse, "lse", _F32, T * att.n_heads), T, n,
        _flat(q_offsets, "q_offsets", _I32, n + 1), _flat(kv_lens, "kv_lens", _I32), table, ld, width, kv, att,
        max_q_hint, ATTEND_PATHS[path], ws.data_ptr(), ws.numel() * ws.element_size(),
        None if err is None else _flat(err, "err", _I32), _on(stream))
    if status:
        check(status, "lora_attend")


class PagedKV:
    """A layer's paged cache: k and v are [page, token, head, dim] tensors (any
    strides with contiguous dims, the same for both), bf16 or float8_e4m3fn (or
    uint8 codes); an e4m3 value is its code times the scale."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        torch = _torch()
        for t, name in ((k, "k"), (v, "v")):
            _dev(t, name)
            if t.dim() != 4 or t.stride(3) != 1 or t.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8):
                raise TypeError(f"{name} must be a bf16 or e4m3 [page, token, head, dim] tensor with contiguous dims")
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must have the same shape, strides and type")
        self.k, self.v = k, v
        self.c = lora_kv_t(k.data_ptr(), v.data_ptr(), *k.shape, *k.stride()[:3],
                           0 if k.dtype == torch.bfloat16 else 1, float(k_scale), float(v_scale))

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv: int, head_dim: int, dtype=None, k_scale: float = 1.0,
              v_scale: float = 1.0, device="cuda") -> "PagedKV":
        """A cache in which the tokens of one head of a page are contiguous."""
        torch = _torch()
        k, v = (torch.empty(n_pages, n_kv, page_size, head_dim, dtype=dtype or torch.bfloat16,
                            device=device).transpose(1, 2) for _ in range(2))
        return cls(k, v, k_scale, v_scale)


class KVStep:
    """Block tables and the per-step arrays of lora_kv_step: room for T rows of
    n_seq requests of up to max_pages pages.  The block table persists over
    steps (it may be replaced by another [n_seq, pages] tensor); ``taken`` is the
    number of pages taken from the front of free_pages.  The other arrays are
    the step's own for its lifetime."""

    _OWN = ("q_offsets", "kv_lens", "positions", "seq_ids", "slot_map", "taken", "err")

    def __init__(self, n_seq: int, T: int, max_pages: int, page_size: int, device="cuda"):
        torch = _torch()
        _types()
        self.page_size, self.n_seq, self.T = int(page_size), int(n_seq), int(T)
        self.block_table = torch.zeros(n_seq, max_pages, dtype=_I32, device=device)
        sizes = dict(q_offsets=n_seq + 1, kv_lens=n_seq, positions=T, seq_ids=T, slot_map=T, taken=1, err=1)
        self._own = tuple(torch.zeros(sizes[k], dtype=_I64 if k == "slot_map" else _I32, device=device)
                          for k in self._OWN)
        self._at = tuple(t.data_ptr() for t in self._own)

    def build(self, ctx_lens, new_lens, free_pages, stream=None) -> None:
        n = self.n_seq
        table, ld, width = _table(self.block_table, n)
        status = load().lora_kv_step(
            _flat(ctx_lens, "ctx_lens", _I32, n), _flat(new_lens, "new_lens", _I32, n), n, self.page_size,
            _flat(free_pages, "free_pages", _I32), free_pages.numel(), table, ld, width, self.T, *self._at, _on(stream))
        if status:
            check(status, "lora_kv_step")


for _i, _name in enumerate(KVStep._OWN):
    setattr(KVStep, _name, property(lambda self, i=_i: self._own[i]))


class Rope:
    """Rotary frequencies of one model on the device."""

    def __init__(self, head_dim: int, rot_dim: Optional[int] = None, theta: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[Mapping] = None, device="cuda"):
        torch = _torch()
        self.rot_dim = int(head_dim if rot_dim is None else rot_dim)
        phases, mscale = lora_rope_phases(self.rot_dim, theta, scaling)
        self.phases = torch.from_numpy(phases.view(np.int64)).to(device)
        self.c = lora_rope_t(self.rot_dim, int(bool(interleaved)), mscale, self.phases.data_ptr())

    def append(self, qkv, q_out, n_heads: int, kv: PagedKV, positions, slot_map, err, stream=None) -> None:
        """q of qkv turned into q_out; k turned, and v, written to kv at slot_map."""
        lora_rope_append(qkv, q_out, n_heads, self.c, positions, slot_map, kv.c, err, stream)


class Attention:
    """One layer's attention over a PagedKV: its parameters, workspace and error
    word.  Layers whose calls do not overlap can share one by passing ``kv``."""

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
        self.ws = torch.zeros(lora_attend_workspace_bytes(self.c, kv.c), dtype=torch.uint8, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def run(self, q, out, q_offsets, kv_lens, block_table, max_q_hint: int = 0, kv: Optional[PagedKV] = None, lse=None,
            path: str = "auto", stream=None) -> None:
        """out = attention of q's rows; max_q_hint is an upper bound on a request's rows (0: taken as T / n_seq)."""
        lora_attend(q, out, q_offsets, kv_lens, block_table, (kv or self.kv).c, self.c, self.ws, self.err, max_q_hint,
                    lse, path, stream)

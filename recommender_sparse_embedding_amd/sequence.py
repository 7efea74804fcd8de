"""Attention over behaviour sequences: binding of the seq_* calls of rse.h.

``SeqAttention`` is a layer's configuration (heads, type, causal or not,
distance boundaries); ``SeqCache`` the paged keys, values and times of every
user's history for serving, one new event a user (seq_attention_step) or
several (seq_attention_chunk) at a time.  Rows are [n_events, heads, dim] tensors whose
last dimension is contiguous; the other strides are free in steps of 16 bytes
(views of a joint projection, for example); only inputs may overlap
themselves (an expanded tensor).  Every call is ordered on the
given stream (default: the current one), and tensors it returns are allocated
for that stream.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import weakref

import torch

from . import BF16, F32, _bytes, _need, _ptr, lib
from ._lib import RseSeqBatch, RseSeqRows, check

_DTYPE = {F32: torch.float32, BF16: torch.bfloat16}


# the current stream's handle without building a stream object (several
# microseconds of a call), where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here(t: torch.Tensor, name: str, stream=None):
    """t: a CUDA tensor (so that the runtime is up)."""
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    if stream is not None and stream.device.index != t.get_device():
        raise ValueError(f"the stream is of {stream.device}, {name} on {t.device}")


def _beside(t: torch.Tensor, other: torch.Tensor, name: str):
    """t: a CUDA tensor on other's device (a kernel would fault on another's memory)."""
    if t.get_device() != other.get_device():
        raise ValueError(f"{name} is on {t.device}, the rows on {other.device}")


def _on(stream):
    """Allocations inside belong to `stream`."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


_PER16 = {torch.float32: 4, torch.bfloat16: 8}


def _rows(t: torch.Tensor, dtype, n: int, heads: int, dim: int, name: str) -> RseSeqRows:
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name}: expected a {dtype} CUDA tensor, got {t.dtype} on {t.device}")
    if t.shape != (n, heads, dim):
        raise ValueError(f"{name}: expected shape ({n}, {heads}, {dim}), got {tuple(t.shape)}")
    row, head, one = t.stride()
    per16 = _PER16[dtype]
    # the stride of a dimension of one element is never used
    if n <= 1:
        row = per16
    if heads == 1:
        head = per16
    p = t.data_ptr()
    if n and (one != 1 or row % per16 or head % per16 or p % 16):
        raise ValueError(f"{name}: the last dimension must be contiguous, and the address and the other strides "
                         f"multiples of 16 bytes (strides {t.stride()})")
    return RseSeqRows(p, row, head)


def _vector(t: torch.Tensor, dtype, n: int, name: str):
    _need(t, dtype, name)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} entries, got {t.numel()}")
    return t.data_ptr()


class SeqAttention:
    """Configuration of attention over behaviour sequences.

    The bias of events i, j is bias[h, number of boundaries <= pos_i - pos_j]
    (ascending int32 boundaries, at most 127); scale defaults to
    1 / sqrt(dim)."""

    def __init__(self, n_heads: int, n_kv_heads: int, dim: int, dtype: int = BF16, boundaries=(),
                 causal: bool = True, scale: float | None = None, device="cuda", stream=None):
        self.n_heads, self.n_kv_heads, self.dim, self.dtype = int(n_heads), int(n_kv_heads), int(dim), dtype
        self.boundaries = [int(b) for b in boundaries]
        if any(not -(2**31) < b < 2**31 for b in self.boundaries):
            raise ValueError("boundaries must lie within int32, above its minimum")
        self.causal, self.scale = bool(causal), float(1.0 / math.sqrt(dim) if scale is None else scale)
        self.device = torch.device(device)
        self.torch_dtype = _DTYPE.get(dtype)
        n = len(self.boundaries)
        arr = (ctypes.c_int32 * max(n, 1))(*self.boundaries)
        sz = ctypes.c_size_t()
        check(lib.rse_seqattn_mem_size(ctypes.byref(sz)), "rse_seqattn_mem_size")
        with _on(stream):
            self.mem = _bytes(sz.value, self.device)
        h = ctypes.c_void_p()
        check(lib.rse_seqattn_create(ctypes.byref(h), _ptr(self.mem), sz.value, self.n_heads, self.n_kv_heads,
                                     self.dim, dtype, int(self.causal), self.scale, arr, n, _stream(stream)),
              "rse_seqattn_create")
        self.handle = h
        self.step_bytes = (-1, -1, 0)            # the last step's batch, max_len and workspace size
        self.chunk_bytes = (None, 0)             # the last chunk's sizes and workspace size
        self._finalizer = weakref.finalize(self, lib.rse_seqattn_destroy, h)

    @property
    def n_buckets(self) -> int:
        return len(self.boundaries) + 1

    def status(self, stream=None) -> int:
        """Sticky status; synchronises the stream."""
        st = ctypes.c_int32()
        check(lib.rse_seqattn_status(self.handle, ctypes.byref(st), _stream(stream)), "rse_seqattn_status")
        return st.value

    def clear_status(self, stream=None):
        check(lib.rse_seqattn_clear_status(self.handle, _stream(stream)), "rse_seqattn_clear_status")


def _size(fn, what: str, *args) -> int:
    sz = ctypes.c_size_t()
    check(fn(*args, ctypes.byref(sz)), what)
    return sz.value


def _on_empty(stream, shape, dtype, device):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _batch(attn: SeqAttention, n: int, pos, bias, seq_offsets, key_off, max_len) -> RseSeqBatch:
    _need(seq_offsets, torch.int64, "seq_offsets")
    if seq_offsets.numel() < 1:
        raise ValueError("seq_offsets must hold batch + 1 entries")
    batch = seq_offsets.numel() - 1
    if n > 0 and batch == 0:
        raise ValueError("events without a sequence: seq_offsets holds one entry only")
    return RseSeqBatch(seq_offsets.data_ptr(), batch, n, n if max_len is None else int(max_len),
                       _vector(pos, torch.int32, n, "pos"),
                       None if key_off is None else _vector(key_off, torch.int64, n, "key_off"),
                       _vector(bias, torch.float32, attn.n_heads * attn.n_buckets, "bias"))


def seq_attention_fwd(attn: SeqAttention, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                      bias: torch.Tensor, seq_offsets: torch.Tensor, key_off: torch.Tensor | None = None,
                      max_len: int | None = None, for_backward: bool = False, out: torch.Tensor | None = None,
                      stream=None):
    """Attention within each sequence of a jagged batch.

    q [n, n_heads, dim], k, v [n, n_kv_heads, dim]; sequence b is events
    seq_offsets[b] .. seq_offsets[b+1] (int64, batch + 1); pos int32 [n] times
    or indexes; bias fp32 [n_heads, n_buckets]; key_off int64 [n]: events whose
    entry is negative (a lookup without a row) are not seen.  max_len: no
    sequence is longer (default: n).  Returns out [n, n_heads, dim], and with
    for_backward also what seq_attention_bwd needs of this call."""
    n = q.shape[0]
    dt, H, D = attn.torch_dtype, attn.n_heads, attn.dim
    args = [_rows(q, dt, n, H, D, "q"), _rows(k, dt, n, attn.n_kv_heads, D, "k"),
            _rows(v, dt, n, attn.n_kv_heads, D, "v")]
    b = _batch(attn, n, pos, bias, seq_offsets, key_off, max_len)
    saved, size = None, 0
    with _on(stream):
        if out is None:
            out = torch.empty((n, H, D), dtype=dt, device=q.device)
        if for_backward:
            size = _size(lib.rse_seqattn_saved_size, "rse_seqattn_saved_size", attn.handle, n, b.max_len)
            saved = _bytes(size, q.device)
    args.append(_rows(out, dt, n, H, D, "out"))
    check(lib.seq_attention_fwd(attn.handle, ctypes.byref(b), *map(ctypes.byref, args), _ptr(saved), size,
                                _stream(stream)), "seq_attention_fwd")
    return (out, saved) if for_backward else out


def seq_attention_bwd(attn: SeqAttention, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                      bias: torch.Tensor, seq_offsets: torch.Tensor, saved: torch.Tensor, dout: torch.Tensor,
                      key_off: torch.Tensor | None = None, max_len: int | None = None, grads=None, stream=None):
    """Gradients (dq, dk, dv, dbias) for the upstream gradient dout
    [n, n_heads, dim]; the other arguments are the forward's, `saved` what it
    returned.  grads: (dq, dk, dv) tensors to write, for example views of one
    joint gradient; dbias is fp32 [n_heads, n_buckets]."""
    n = q.shape[0]
    dt, H, Hk, D = attn.torch_dtype, attn.n_heads, attn.n_kv_heads, attn.dim
    b = _batch(attn, n, pos, bias, seq_offsets, key_off, max_len)
    _need(saved, torch.uint8, "saved")
    with _on(stream):
        dq, dk, dv = grads if grads is not None else (
            torch.empty((n, h, D), dtype=dt, device=q.device) for h in (H, Hk, Hk))
        dbias = torch.empty((H, attn.n_buckets), dtype=torch.float32, device=q.device)
        size = _size(lib.rse_seqattn_bwd_workspace_size, "rse_seqattn_bwd_workspace_size", attn.handle, n, b.batch,
                     b.max_len)
        ws = _bytes(size, q.device)
    rows = [_rows(t, dt, n, h, D, name) for t, h, name in (
        (q, H, "q"), (k, Hk, "k"), (v, Hk, "v"), (dout, H, "dout"), (dq, H, "dq"), (dk, Hk, "dk"), (dv, Hk, "dv"))]
    ref = [ctypes.byref(r) for r in rows]
    check(lib.seq_attention_bwd(attn.handle, ctypes.byref(b), *ref[:3], _ptr(saved), saved.numel(), *ref[3:],
                                _ptr(dbias), _ptr(ws), ws.numel(), _stream(stream)), "seq_attention_bwd")
    return dq, dk, dv, dbias


# ------------------------------------------------------------------- cache --
class SeqCache:
    """Paged keys, values and times of users' histories: k, v
    [n_pages, page_size, n_kv_heads, dim], pos int32 [n_pages, page_size]
    (the caller's tensors; page_size a power of two in 8 .. 1024)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, stream=None):
        dtype = {t: d for d, t in _DTYPE.items()}.get(k.dtype)
        if dtype is None or k.dim() != 4:
            raise TypeError("k: expected a fp32 or bf16 [n_pages, page_size, n_kv_heads, dim] tensor")
        for t, dt, name in ((k, k.dtype, "k"), (v, k.dtype, "v"), (pos, torch.int32, "pos")):
            _need(t, dt, name)
        if v.shape != k.shape or pos.shape != k.shape[:2]:
            raise ValueError("v must have the shape of k, and pos its first two dimensions")
        self.k, self.v, self.pos, self.dtype = k, v, pos, dtype
        self.n_pages, self.page_size, self.n_kv_heads, self.dim = k.shape
        self.device = k.device
        size = _size(lib.rse_seqcache_meta_size, "rse_seqcache_meta_size")
        with _on(stream):
            self.meta = _bytes(size, self.device)
        h = ctypes.c_void_p()
        check(lib.rse_seqcache_create(ctypes.byref(h), _ptr(self.meta), size, _ptr(k), _ptr(v), _ptr(pos),
                                      self.n_pages, self.page_size, self.n_kv_heads, self.dim, dtype,
                                      _stream(stream)), "rse_seqcache_create")
        self.handle = h
        self._finalizer = weakref.finalize(self, lib.rse_seqcache_destroy, h)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, dim: int, dtype: int = BF16, device="cuda",
              stream=None) -> "SeqCache":
        """A cache over new memory (not cleared: no call reads what none wrote)."""
        with _on(stream):
            k, v = (torch.empty((n_pages, page_size, n_kv_heads, dim), dtype=_DTYPE[dtype], device=device)
                    for _ in range(2))
            pos = torch.empty((n_pages, page_size), dtype=torch.int32, device=device)
        return cls(k, v, pos, stream)

    def status(self, stream=None) -> int:
        """Sticky status; synchronises the stream."""
        st = ctypes.c_int32()
        check(lib.rse_seqcache_status(self.handle, ctypes.byref(st), _stream(stream)), "rse_seqcache_status")
        return st.value

    def clear_status(self, stream=None):
        check(lib.rse_seqcache_clear_status(self.handle, _stream(stream)), "rse_seqcache_clear_status")


def _table(page_table: torch.Tensor, batch: int) -> int:
    _need(page_table, torch.int32, "page_table")
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError(f"page_table must be [{batch}, max_pages], got {tuple(page_table.shape)}")
    return page_table.shape[1]


def seq_cache_assign(cache: SeqCache, counts: torch.Tensor, lens: torch.Tensor, page_table: torch.Tensor,
                     free_pages: torch.Tensor, n_events: int, stream=None):
    """Pages and slots of counts[b] new events after the lens[b] cached of user
    b (int64 [batch]).  page_table int32 [batch, max_pages] gets the pages,
    taken in order from free_pages (int32).  Returns (slots int64 [n_events],
    seq_offsets int64 [batch + 1], taken int64 [1]); n_events is the counts'
    sum.  cache.status() tells of a free list that was too short, and of pages
    outside the pool, whose events get slot -1."""
    batch = counts.numel()
    _need(counts, torch.int64, "counts")
    lens_p = _vector(lens, torch.int64, batch, "lens")
    max_pages = _table(page_table, batch)
    _need(free_pages, torch.int32, "free_pages")
    with _on(stream):
        new = lambda n: torch.empty(n, dtype=torch.int64, device=counts.device)  # noqa: E731
        slots, offsets, taken = new(int(n_events)), new(batch + 1), new(1)
        ws = _bytes(_size(lib.rse_seqcache_assign_workspace_size, "rse_seqcache_assign_workspace_size", batch),
                    counts.device)
    check(lib.seq_cache_assign(cache.handle, _ptr(counts), lens_p, batch, _ptr(page_table), max_pages,
                               _ptr(free_pages), free_pages.numel(), int(n_events), _ptr(slots), _ptr(offsets),
                               _ptr(taken), _ptr(ws), ws.numel(), _stream(stream)), "seq_cache_assign")
    return slots, offsets, taken


def seq_cache_write(cache: SeqCache, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                    stream=None):
    """Store k, v [n, n_kv_heads, dim] and pos int32 [n] at their slots
    (int64 [n]; negative: skipped)."""
    n, dt = k.shape[0], cache.k.dtype
    slots_p, pos_p = _vector(slots, torch.int64, n, "slots"), _vector(pos, torch.int32, n, "pos")
    kr, vr = (_rows(t, dt, n, cache.n_kv_heads, cache.dim, name) for t, name in ((k, "k"), (v, "v")))
    check(lib.seq_cache_write(cache.handle, slots_p, n, ctypes.byref(kr), ctypes.byref(vr), pos_p, _stream(stream)),
          "seq_cache_write")


def seq_attention_step(attn: SeqAttention, cache: SeqCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       pos: torch.Tensor, bias: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                       max_len: int | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One new event per user: stores its k, v [batch, n_kv_heads, dim] and pos
    int32 [batch] as event lens[b] (int64; negative: idle) and returns its
    attention [batch, n_heads, dim] over the whole history, itself included.
    max_len: no history with its new event is longer (default: the table's
    width).  lens is not changed.  There is no key_off here: events that
    seq_attention_fwd would hide are kept out of the cache."""
    batch = q.shape[0]
    dt, H, Hk, D = attn.torch_dtype, attn.n_heads, attn.n_kv_heads, attn.dim
    args = [_rows(q, dt, batch, H, D, "q"), _rows(k, dt, batch, Hk, D, "k"), _rows(v, dt, batch, Hk, D, "v")]
    max_pages = _table(page_table, batch)
    most = max_pages * cache.page_size if max_len is None else int(max_len)
    pos_p = _vector(pos, torch.int32, batch, "pos")
    bias_p = _vector(bias, torch.float32, H * attn.n_buckets, "bias")
    lens_p = _vector(lens, torch.int64, batch, "lens")
    known = attn.step_bytes
    if known[:2] == (batch, most):
        size = known[2]
    else:
        size = _size(lib.rse_seqattn_step_workspace_size, "rse_seqattn_step_workspace_size", attn.handle, batch, most)
        attn.step_bytes = (batch, most, size)
    if out is None:
        out = _on_empty(stream, (batch, H, D), dt, q.device)
    ws = _on_empty(stream, size, torch.uint8, q.device) if size else None
    o = _rows(out, dt, batch, H, D, "out")
    byref = ctypes.byref
    check(lib.seq_attention_step(attn.handle, cache.handle, byref(args[0]), byref(args[1]), byref(args[2]), pos_p,
                                 bias_p, page_table.data_ptr(), max_pages, lens_p, batch, most, byref(o), _ptr(ws),
                                 size, _stream(stream)), "seq_attention_step")
    return out


def seq_attention_chunk(attn: SeqAttention, cache: SeqCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        pos: torch.Tensor, bias: torch.Tensor, seq_offsets: torch.Tensor, page_table: torch.Tensor,
                        lens: torch.Tensor, max_new: int | None = None, max_len: int | None = None,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Several new events per user: events seq_offsets[b] .. seq_offsets[b+1]
    (int64, batch + 1) of q [n, n_heads, dim], k, v [n, n_kv_heads, dim] and pos
    int32 [n] are user b's, stored as events lens[b] and on (int64 [batch];
    negative: idle).  Returns their attention [n, n_heads, dim] over the history
    and each other (a causal handle: up to themselves).  max_new: no user has
    more new events (default: n); max_len: no history with them is longer
    (default: the table's width).  lens is not changed, and there is no key_off,
    as in seq_attention_step."""
    n = q.shape[0]
    dt, H, Hk, D = attn.torch_dtype, attn.n_heads, attn.n_kv_heads, attn.dim
    args = [_rows(q, dt, n, H, D, "q"), _rows(k, dt, n, Hk, D, "k"), _rows(v, dt, n, Hk, D, "v")]
    _here(q, "q", stream)
    b = _batch(attn, n, pos, bias, seq_offsets, None, max_new)
    batch = b.batch
    max_pages = _table(page_table, batch)
    lens_p = _vector(lens, torch.int64, batch, "lens")
    # (one comparison where they agree: the names only when they do not)
    if not (q.get_device() == k.get_device() == v.get_device() == pos.get_device() == bias.get_device()
            == seq_offsets.get_device() == page_table.get_device() == lens.get_device() == cache.k.get_device()
            == attn.mem.get_device()):
        for t, name in ((k, "k"), (v, "v"), (pos, "pos"), (bias, "bias"), (seq_offsets, "seq_offsets"), (lens, "lens"),
                        (page_table, "page_table"), (cache.k, "cache"), (attn.mem, "attn")):
            _beside(t, q, name)
    most = max_pages * cache.page_size if max_len is None else int(max_len)
    shape = (n, batch, b.max_len, most)
    known = attn.chunk_bytes
    if known[0] == shape:
        size = known[1]
    else:
        size = _size(lib.rse_seqattn_chunk_workspace_size, "rse_seqattn_chunk_workspace_size", attn.handle, *shape)
        attn.chunk_bytes = (shape, size)
    if out is None:
        out = _on_empty(stream, (n, H, D), dt, q.device)
        o = RseSeqRows(out.data_ptr(), H * D, D)
    else:
        o = _rows(out, dt, n, H, D, "out")
        _beside(out, q, "out")
    ws = _on_empty(stream, size, torch.uint8, q.device) if size else None
    byref = ctypes.byref
    check(lib.seq_attention_chunk(attn.handle, cache.handle, byref(b), byref(args[0]), byref(args[1]), byref(args[2]),
                                  page_table.data_ptr(), max_pages, lens_p, most, byref(o), _ptr(ws), size,
                                  _stream(stream)), "seq_attention_chunk")
    return out

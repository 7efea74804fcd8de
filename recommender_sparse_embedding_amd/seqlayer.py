"""The layer around the sequence attention: binding of the layer norm and of
the gated feed-forward's projections of rse.h.

Rows are [n, width] tensors whose last dimension is contiguous; the distance
between rows is free (for the gated calls in steps of 16 bytes), so slices of
wider tensors and expanded inputs will do.  Every call is ordered on the given
stream (default: the current one) of the current device, where all its tensors
are, and tensors it returns are allocated for that stream.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import BF16, F32, SILU, _bytes, _ptr, lib
from ._lib import RseSeqMat, check
from .sequence import _PER16, _beside, _here, _on, _on_empty, _size, _stream, _vector

_KIND = {torch.float32: F32, torch.bfloat16: BF16}


def _kind(x: torch.Tensor, name: str, stream) -> int:
    kind = _KIND.get(x.dtype)
    if kind is None or not x.is_cuda or x.dim() != 2:
        raise TypeError(f"{name}: expected a fp32 or bf16 [n, width] CUDA tensor, got {x.dtype} {tuple(x.shape)} on {x.device}")
    _here(x, name, stream)
    return kind


def _new(x: torch.Tensor, n: int, width: int, stream):
    """A tensor of x's type for a result, and its description (a call of a few
    rows takes as long here as on the GPU, so what is known is not looked at)."""
    if stream is None:
        t = x.new_empty((n, width))
    else:
        with torch.cuda.stream(stream):
            t = x.new_empty((n, width))
    return t, RseSeqMat(t.data_ptr(), width)


def _mat(t: torch.Tensor, like: torch.Tensor, n: int, width: int, name: str, per: int = 1) -> RseSeqMat:
    """per: elements that address and stride are multiples of."""
    if t.dtype != like.dtype or t.get_device() != like.get_device():
        raise TypeError(f"{name}: expected a {like.dtype} tensor on {like.device}, got {t.dtype} on {t.device}")
    if t.shape != (n, width):
        raise ValueError(f"{name}: expected shape ({n}, {width}), got {tuple(t.shape)}")
    row, one = t.stride()
    if n <= 1:                  # the stride of a dimension of one element is never used
        row = 0
    p = t.data_ptr()
    if n and ((one != 1 and width > 1) or row % per or (per > 1 and p % 16)):
        raise ValueError(f"{name}: the last dimension must be contiguous"
                         + (", and the address and the row stride multiples of 16 bytes" if per > 1 else "")
                         + f" (strides {t.stride()})")
    return RseSeqMat(p, row)


def _floats(t: torch.Tensor | None, like: torch.Tensor, n: int, name: str):
    if t is None:
        return None
    p = _vector(t, torch.float32, n, name)
    _beside(t, like, name)
    return p


def _ref(m: RseSeqMat | None):
    return None if m is None else ctypes.byref(m)


# workspace sizes, by sizes alone
@functools.lru_cache(maxsize=64)
def _norm_bytes(n: int, dim: int, kind: int) -> int:
    return _size(lib.rse_seq_layer_norm_bwd_workspace_size, "rse_seq_layer_norm_bwd_workspace_size", n, dim, kind)


@functools.lru_cache(maxsize=64)
def _gated_bytes(n: int, dim: int, hidden: int, kind: int) -> int:
    return _size(lib.rse_seq_gated_linear_bwd_workspace_size, "rse_seq_gated_linear_bwd_workspace_size", n, dim, hidden, kind)


class LayerNormOut(NamedTuple):
    y: torch.Tensor
    sum: torch.Tensor | None         # x + residual as stored; None without a residual
    stats: torch.Tensor | None       # fp32 [n, 2], for the backward; None unless asked for


def seq_layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None, bias: torch.Tensor | None, eps: float = 1e-5,
                       residual: torch.Tensor | None = None, for_backward: bool = False, out: torch.Tensor | None = None,
                       sum_out: torch.Tensor | None = None, stream=None) -> LayerNormOut:
    """Layer norm of the rows of x [n, dim], or with residual of x + residual as
    it is stored (the stream that later layers and the backward read; sum_out:
    a tensor to write it to, x or residual for example).  weight, bias: fp32
    [dim] or None (1 and 0)."""
    kind = _kind(x, "x", stream)
    n, dim = x.shape
    xm = _mat(x, x, n, dim, "x")
    wp, bp = _floats(weight, x, dim, "weight"), _floats(bias, x, dim, "bias")
    if residual is None and sum_out is not None:
        raise ValueError("sum_out is given without a residual")
    if out is None:
        out, ym = _new(x, n, dim, stream)
    else:
        ym = _mat(out, x, n, dim, "out")
    rm = sm = None
    if residual is not None:
        rm = _mat(residual, x, n, dim, "residual")
        if sum_out is None:
            sum_out, sm = _new(x, n, dim, stream)
        else:
            sm = _mat(sum_out, x, n, dim, "sum_out")
    stats = _on_empty(stream, (n, 2), torch.float32, x.device) if for_backward else None
    check(lib.seq_layer_norm_fwd(_ref(xm), _ref(rm), _ref(sm), wp, bp, eps, n, dim, kind, _ref(ym), _ptr(stats),
                                 _stream(stream)), "seq_layer_norm_fwd")
    return LayerNormOut(out, sum_out, stats)


def seq_layer_norm_bwd(x: torch.Tensor, dy: torch.Tensor, weight: torch.Tensor | None, stats: torch.Tensor,
                       dsum: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """(dx, dweight, dbias) for the upstream gradient dy of y.  x: the rows that
    were normalised (the forward's x, or its sum); stats: the forward's.  dsum:
    the gradient that reaches the sum by the stream; dx is then the gradient of
    x and of the residual.  dweight, dbias: fp32 [dim]."""
    kind = _kind(x, "x", stream)
    n, dim = x.shape
    xm, dym = _mat(x, x, n, dim, "x"), _mat(dy, x, n, dim, "dy")
    wp, sp = _floats(weight, x, dim, "weight"), _floats(stats, x, 2 * n, "stats")
    dsm = None if dsum is None else _mat(dsum, x, n, dim, "dsum")
    with _on(stream):
        dw, db = (torch.empty(dim, dtype=torch.float32, device=x.device) for _ in range(2))
        ws = _bytes(_norm_bytes(n, dim, kind), x.device)
    if out is None:
        out, dxm = _new(x, n, dim, stream)
    else:
        dxm = _mat(out, x, n, dim, "out")
    check(lib.seq_layer_norm_bwd(_ref(xm), _ref(dym), wp, sp, _ref(dsm), n, dim, kind, _ref(dxm), _ptr(dw), _ptr(db),
                                 _ptr(ws), ws.numel(), _stream(stream)), "seq_layer_norm_bwd")
    return out, dw, db


def _gated(x, w_gate, w_up, stream):
    kind = _kind(x, "x", stream)
    n, dim = x.shape
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate: expected [hidden, dim], got {tuple(w_gate.shape)}")
    hidden, per = w_gate.shape[0], _PER16[x.dtype]
    return kind, n, dim, hidden, per, [_mat(x, x, n, dim, "x", per), _mat(w_gate, x, hidden, dim, "w_gate", per),
                                       _mat(w_up, x, hidden, dim, "w_up", per)]


def seq_gated_linear_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: int = SILU,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """act(x w_gate^T) (x w_up^T) [n, hidden] for x [n, dim] and w_gate, w_up
    [hidden, dim] of one type; dim and hidden are multiples of 16 bytes.  act:
    SIGMOID, SILU or GELU."""
    kind, n, dim, hidden, per, mats = _gated(x, w_gate, w_up, stream)
    if out is None:
        out, o = _new(x, n, hidden, stream)
    else:
        o = _mat(out, x, n, hidden, "out", per)
    check(lib.seq_gated_linear_fwd(*map(_ref, mats), n, dim, hidden, kind, act, _ref(o), _stream(stream)),
          "seq_gated_linear_fwd")
    return out


def seq_gated_linear_bwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, dout: torch.Tensor, act: int = SILU,
                         grads=None, stream=None):
    """(dx, dw_gate, dw_up) for the upstream gradient dout [n, hidden]; the other
    arguments are the forward's, which leaves nothing else for this call.
    grads: tensors to write them to (halves of one joint gradient, for example)."""
    kind, n, dim, hidden, per, mats = _gated(x, w_gate, w_up, stream)
    mats.append(_mat(dout, x, n, hidden, "dout", per))
    shapes = ((n, dim), (hidden, dim), (hidden, dim))
    with _on(stream):
        if grads is None:
            grads = tuple(torch.empty(s, dtype=x.dtype, device=x.device) for s in shapes)
        ws = _bytes(_gated_bytes(n, dim, hidden, kind), x.device)
    mats += [_mat(t, x, *s, name, per) for t, s, name in zip(grads, shapes, ("dx", "dw_gate", "dw_up"))]
    check(lib.seq_gated_linear_bwd(*map(_ref, mats[:4]), n, dim, hidden, kind, act, *map(_ref, mats[4:]), _ptr(ws), ws.numel(),
                                   _stream(stream)), "seq_gated_linear_bwd")
    return tuple(grads)

"""What lies between a layer's linear products: embedding, dropout, and the norm with the residual's addition.

Like mx4.py and mx8.py these record no autograd graph: each forward call has
its backward call beside it.  The table's and the norm's weight gradients go
straight into a rank's 16-bit gradient row (a view of it, as MuonBuffers.matrix
gives), the table's also on top of what is there; the linear layers' calls
return theirs, to be copied.  A norm's weight that does not start on 16 bytes
costs its calls up to twice the time.  Inputs whose
gradient autograd is to find are refused, and inputs with forward-mode tangents.  Activations are [..., cols] with
contiguous rows.  Everything here runs on torch's current stream of the
tensors' device, where the tensors it makes belong.
"""

from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _binding as B
from .mx4 import Mx4Matrix, MxMatrix, _at, _dtype, _rows, _same_gpu
from .mx8 import Mx8Matrix


class Norm(NamedTuple):
    """What rms_norm gives: the new stream, its norm in 16 bits, and in microscaled ones (None for what was not asked)."""
    h: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    q: Optional[MxMatrix]


def _plain(name: str, *tensors: Optional[torch.Tensor]) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise B.ZeroError(1, f"{name} records no autograd graph: pass detached tensors (or call it under torch.no_grad()) "
                             f"and take the gradients from the backward call")


def _matrix(t: torch.Tensor) -> torch.Tensor:
    """[..., cols] as [rows, cols], without a copy."""
    if t.dim() == 2:
        return t
    if t.dim() < 1:
        raise B.ZeroError(1, "expected a tensor of at least one dimension")
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(t.shape[:-1].numel(), t.shape[-1])
    except RuntimeError as e:
        raise B.ZeroError(1, f"expected contiguous rows at one distance, got the shape {tuple(t.shape)} with the strides "
                             f"{t.stride()}") from e


def _like(t: torch.Tensor, *others: Tuple[str, Optional[torch.Tensor]]) -> None:
    for name, o in others:
        if o is not None and (o.shape != t.shape or o.dtype != t.dtype):
            raise B.ZeroError(1, f"{name} must be {tuple(t.shape)} of {t.dtype}, got {tuple(o.shape)} of {o.dtype}")


def _spec_gpu(dropout: Optional[B.Dropout]) -> Tuple[torch.Tensor, ...]:
    step = getattr(dropout, "tensor", None)
    if step is None or isinstance(step, int):
        return ()
    if step.dtype != torch.int64 or step.numel() < 1:
        raise B.ZeroError(1, "step must be a tensor of one int64")
    return (step,)


def _vector(name: str, v: torch.Tensor, cols: int, dtype) -> torch.Tensor:
    if v.dim() != 1 or v.shape[0] != cols or v.dtype != dtype or (cols > 1 and v.stride(0) != 1):
        raise B.ZeroError(1, f"{name} must be {cols} contiguous values of {dtype}, got {tuple(v.shape)} of {v.dtype}")
    return v


def _room(workspace: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if not workspace.is_contiguous():
        raise B.ZeroError(1, "workspace must be contiguous")
    return workspace


# --------------------------------------------------------------- embedding
def _table(name: str, ids: torch.Tensor, table: torch.Tensor) -> torch.Tensor:
    if ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise B.ZeroError(1, f"ids must be a contiguous tensor of int32 or int64, got {ids.dtype}")
    if table.dim() != 2 or table.shape[0] < 1:
        raise B.ZeroError(1, f"{name} must be a matrix of at least one row, got {tuple(table.shape)}")
    return table


def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids], [*ids.shape, dim]; an id outside the table is padding and gives zeros."""
    _plain("embedding", table, out)
    _table("table", ids, table)
    vocab, dim = table.shape
    if out is None:
        out = torch.empty((*ids.shape, dim), dtype=table.dtype, device=table.device)
    elif out.shape != (*ids.shape, dim) or out.dtype != table.dtype:
        raise B.ZeroError(1, f"out must be {(*ids.shape, dim)} of {table.dtype}")
    _same_gpu(table, ids, out)
    o = _matrix(out)
    with _at(table):
        B.zero_embedding(_dtype(table), vocab, dim, table, ids.numel(), ids, o, scale, ld_table=_rows(table), ld_out=_rows(o))
    return out


def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, dtable: torch.Tensor, scale: float = 1.0,
                       accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient into dtable [vocab, dim], every row of it (with accumulate, added to what it holds).
    workspace: zero_embedding_backward_workspace_bytes(vocab, dim, tokens) bytes to reuse from call to call."""
    _plain("embedding_backward", dout, dtable)
    _table("dtable", ids, dtable)
    vocab, dim = dtable.shape
    if dout.shape != (*ids.shape, dim) or dout.dtype != dtable.dtype:
        raise B.ZeroError(1, f"dout must be {(*ids.shape, dim)} of {dtable.dtype}, got {tuple(dout.shape)} of {dout.dtype}")
    _same_gpu(dtable, ids, dout)
    g = _matrix(dout)
    with _at(dtable):
        room = _room(workspace, B.zero_embedding_backward_workspace_bytes(vocab, dim, ids.numel()), dtable.device)
        _same_gpu(dtable, room)
        B.zero_embedding_backward(_dtype(dtable), vocab, dim, g, ids.numel(), ids, dtable, room, scale, accumulate,
                                  ld_dout=_rows(g), ld_dtable=_rows(dtable))
    return dtable


# ----------------------------------------------------------------- dropout
def dropout(x: torch.Tensor, spec: B.Dropout, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with spec's dropout (dropout_spec); the same call on the output's gradient is the backward pass.
    out may be x."""
    _plain("dropout", x, out)
    out = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else out
    _like(x, ("out", out))
    a, o = _matrix(x), _matrix(out)
    _same_gpu(x, out, *_spec_gpu(spec))
    with _at(x):
        B.zero_dropout(_dtype(x), a.shape[0], a.shape[1], a, o, spec, ld_src=_rows(a), ld_out=_rows(o))
    return out


# -------------------------------------------------------------------- norm
def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
             dropout: Optional[B.Dropout] = None, bits: int = 0, wide: bool = True, out: Optional[MxMatrix] = None) -> Norm:
    """The stream h = residual + dropout(x) and its norm: in 16 bits (wide), and in microscaled 8 or 4 bits (bits), as
    mx8_linear and mx4_product take it.  Without residual and dropout the stream is x itself, and h is x.
    out: a Mx8Matrix or Mx4Matrix of x's size to reuse from call to call."""
    _plain("rms_norm", x, weight, residual)
    if bits not in (0, 4, 8):
        raise B.ZeroError(1, f"bits must be 0, 4 or 8, got {bits}")
    _like(x, ("residual", residual))
    a = _matrix(x)
    rows, cols = a.shape
    _vector("weight", weight, cols, x.dtype)
    kind = {0: None, 4: Mx4Matrix, 8: Mx8Matrix}[bits]
    if out is not None and (kind is None or not isinstance(out, kind) or (out.rows, out.cols) != (rows, cols)):
        raise B.ZeroError(1, f"out must be a matrix of {rows} x {cols} in {bits} bits")
    _same_gpu(x, weight, *(() if residual is None else (residual,)), *(() if out is None else (out.codes, out.scales)),
              *_spec_gpu(dropout))
    h = x if residual is None and dropout is None else torch.empty_like(x, memory_format=torch.contiguous_format)
    y = torch.empty_like(x, memory_format=torch.contiguous_format) if wide else None
    q = None if kind is None else kind(rows, cols, device=x.device) if out is None else out
    r = None if residual is None else _matrix(residual)
    if h is x and y is None and q is None:
        raise B.ZeroError(1, "there is nothing to write: neither wide nor bits")
    with _at(x):
        B.zero_rms_norm(_dtype(x), rows, cols, a, weight, eps, residual16=r, h16=None if h is x else h, out16=y, bits=bits,
                        codes=None if q is None else q.codes, scales=None if q is None else q.scales, dropout=dropout,
                        ld_x=_rows(a), ld_residual=None if r is None else _rows(r))
    return Norm(h, y, q)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                      dh_in: Optional[torch.Tensor] = None, dropout: Optional[B.Dropout] = None,
                      dweight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dresidual, dx, dweight) from the gradient of the norm's output and that of the stream from elsewhere (dh_in).
    Without dropout dx is dresidual.  dweight: where to put the weight's gradient; workspace:
    zero_rms_norm_backward_workspace_bytes(rows, cols) bytes to reuse from call to call."""
    _plain("rms_norm_backward", dy, h, weight, dh_in, dweight)
    _like(h, ("dy", dy), ("dh_in", dh_in))
    g, s = _matrix(dy), _matrix(h)
    rows, cols = s.shape
    _vector("weight", weight, cols, h.dtype)
    if dweight is None:
        dweight = torch.empty(cols, dtype=h.dtype, device=h.device)
    _vector("dweight", dweight, cols, h.dtype)
    _same_gpu(h, dy, weight, dweight, *(() if dh_in is None else (dh_in,)), *_spec_gpu(dropout))
    dh = torch.empty_like(h, memory_format=torch.contiguous_format)
    dx = None if dropout is None else torch.empty_like(dh)
    i = None if dh_in is None else _matrix(dh_in)
    with _at(h):
        room = _room(workspace, B.zero_rms_norm_backward_workspace_bytes(rows, cols), h.device)
        _same_gpu(h, room)
        B.zero_rms_norm_backward(_dtype(h), rows, cols, g, s, weight, eps, dh, room, dh_in16=i, dx16=dx, dweight16=dweight,
                                 dropout=dropout, ld_dy=_rows(g), ld_h=_rows(s), ld_in=None if i is None else _rows(i))
    return dh, dh if dx is None else dx, dweight

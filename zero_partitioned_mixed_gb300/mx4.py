"""Matrices in microscaled 4-bit floats, and linear layers on them (mx8.py has those in 8 bits).

A rank that holds its parameters in 4 bits multiplies with the codes as they
are; the three products of a layer's training step are one call on
operands quantised along the dimension that is summed over.  Everything here
runs on torch's current stream of the tensors' device, where the tensors it
makes belong.
"""

from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import _binding as B

_ZDT = {torch.float16: B.ZERO_FP16, torch.bfloat16: B.ZERO_BF16}


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _ZDT:
        raise B.ZeroError(1, f"expected fp16 or bf16, got {t.dtype}")
    return _ZDT[t.dtype]


def _same_gpu(*tensors: torch.Tensor) -> None:
    # A tangent of forward-mode differentiation lies beside a tensor, whatever requires_grad and the grad mode say; the calls
    # see the values alone.  There are none outside a dual level, where asking for them (0.6 us a tensor) is left out.
    if getattr(forward_ad, "_current_level", 0) >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise B.ZeroError(1, "a tensor has a forward-mode tangent, which would be lost: pass detached tensors")
    for t in tensors:
        if not t.is_cuda or t.device != tensors[0].device:
            raise B.ZeroError(1, f"expected tensors on one GPU, got {[str(x.device) for x in tensors]}")


def _at(t: torch.Tensor):
    """The tensor's device as the current one, for a call and for its stream."""
    return contextlib.nullcontext() if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def _rows(t: torch.Tensor) -> int:
    """The leading dimension of a 2-D tensor whose rows are contiguous and do not
    share memory (an expanded tensor's do: make it contiguous first)."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise B.ZeroError(1, f"expected a 2-D tensor with contiguous rows, got the shape {tuple(t.shape)} "
                             f"with the strides {t.stride()}")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class MxMatrix:
    """Codes and scales of a rows x cols matrix, in the library's layout; Mx4Matrix and mx8.Mx8Matrix say in which width."""

    bits = 0

    def __init__(self, rows: int, cols: int, device="cuda"):
        self.rows, self.cols = rows, cols
        self.codes = torch.empty(max(16, self._codes_bytes(rows, cols)), dtype=torch.uint8, device=device)
        self.scales = torch.empty(max(16, self._scales_bytes(rows, cols)), dtype=torch.uint8, device=device)

    @classmethod
    def of(cls, src: torch.Tensor, transpose: bool = False) -> "MxMatrix":
        r, c = src.shape
        return cls(*((c, r) if transpose else (r, c)), device=src.device).fill(src, transpose)

    def fill(self, src: torch.Tensor, transpose: bool = False) -> "MxMatrix":
        """Quantise src along its rows, or along its columns (then self holds its transpose)."""
        r, c = src.shape
        if ((c, r) if transpose else (r, c)) != (self.rows, self.cols):
            raise B.ZeroError(1, f"expected a matrix for {self.rows} x {self.cols}, got {tuple(src.shape)}")
        _same_gpu(src, self.codes, self.scales)
        with _at(src):
            self._quantize(_dtype(src), r, c, src, self.codes, self.scales, ld=_rows(src), transpose=transpose)
        return self

    def values(self, dtype=torch.bfloat16) -> torch.Tensor:
        _same_gpu(self.codes, self.scales)
        out = torch.empty((self.rows, self.cols), dtype=dtype, device=self.codes.device)
        with _at(out):
            self._dequantize(_dtype(out), self.rows, self.cols, self.codes, self.scales, out)
        return out

    @classmethod
    def product(cls, a: "MxMatrix", b: "MxMatrix", dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """a b^T, both quantised along the dimension that is summed over."""
        for m in (a, b):
            if not isinstance(m, cls):
                raise B.ZeroError(1, f"expected a {cls.__name__}, got a {type(m).__name__}")
        if a.cols != b.cols:
            raise B.ZeroError(1, f"the operands have {a.cols} and {b.cols} columns")
        if out is None:
            out = torch.empty((a.rows, b.rows), dtype=dtype, device=a.codes.device)
        elif tuple(out.shape) != (a.rows, b.rows):
            raise B.ZeroError(1, f"out must be {a.rows} x {b.rows}")
        _same_gpu(out, a.codes, a.scales, b.codes, b.scales)
        with _at(out):
            cls._matmul(_dtype(out), a.rows, b.rows, a.cols, a.codes, a.scales, b.codes, b.scales, out, ld=_rows(out))
        return out


class Mx4Matrix(MxMatrix):
    bits = 4
    _codes_bytes, _scales_bytes = staticmethod(B.zero_mx4_codes_bytes), staticmethod(B.zero_mx4_scales_bytes)
    _quantize, _dequantize = staticmethod(B.zero_mx4_quantize), staticmethod(B.zero_mx4_dequantize)
    _matmul = staticmethod(B.zero_mx4_matmul)


def mx4_product(a: Mx4Matrix, b: Mx4Matrix, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a b^T, both quantised along the dimension that is summed over."""
    return Mx4Matrix.product(a, b, dtype, out)


def mx4_linear(x: torch.Tensor, w: Mx4Matrix, out: Optional[torch.Tensor] = None,
               scratch: Optional[Mx4Matrix] = None) -> torch.Tensor:
    """y = x w^T: x [tokens, inner] in 16 bits is quantised, w [outer, inner] is kept in 4.
    scratch: a Mx4Matrix of x's size to reuse from call to call.
    The call records no autograd graph (mx4_linear_backward gives the gradients),
    so an x whose gradient autograd is to find is refused, and one with a forward-mode tangent."""
    if x.requires_grad and torch.is_grad_enabled():
        raise B.ZeroError(1, "mx4_linear records no autograd graph: pass x.detach() (or call it under torch.no_grad()) "
                             "and take the gradients from mx4_linear_backward")
    q = scratch.fill(x) if scratch is not None else Mx4Matrix.of(x)
    return mx4_product(q, w, x.dtype, out)


def mx4_linear_backward(dy: torch.Tensor, x: torch.Tensor, w_t: Mx4Matrix) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of y = x w^T, with the rounding of the operands passed through:
    dx = dy w and dw = dy^T x, each from operands quantised along the summed
    dimension.  w_t: w quantised along its columns (Mx4Matrix.of(w, transpose=True)).
    Both are new matrices, constants to autograd whatever dy and x require."""
    dx = mx4_product(Mx4Matrix.of(dy), w_t, dy.dtype)
    dw = mx4_product(Mx4Matrix.of(dy, True), Mx4Matrix.of(x, True), dy.dtype)
    return dx, dw

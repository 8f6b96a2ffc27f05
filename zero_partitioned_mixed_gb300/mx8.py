"""Matrices in microscaled 8-bit floats (e4m3 elements), and linear layers on them.

The same calls as mx4.py's, for layers that 4 bits are too coarse for.  The
norm of layers.py writes its result in these codes, so that the product after
it reads them as they are.  Everything here runs on torch's current stream of
the tensors' device, where the tensors it makes belong.
"""

from __future__ import annotations

from typing import Optional, Tuple, Union

import torch

from . import _binding as B
from .mx4 import MxMatrix


class Mx8Matrix(MxMatrix):
    bits = 8
    _codes_bytes, _scales_bytes = staticmethod(B.zero_mx8_codes_bytes), staticmethod(B.zero_mx8_scales_bytes)
    _quantize, _dequantize = staticmethod(B.zero_mx8_quantize), staticmethod(B.zero_mx8_dequantize)
    _matmul = staticmethod(B.zero_mx8_matmul)


def mx8_product(a: Mx8Matrix, b: Mx8Matrix, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a b^T, both quantised along the dimension that is summed over."""
    return Mx8Matrix.product(a, b, dtype, out)


def mx8_linear(x: Union[torch.Tensor, Mx8Matrix], w: Mx8Matrix, out: Optional[torch.Tensor] = None,
               scratch: Optional[Mx8Matrix] = None, dtype=torch.bfloat16) -> torch.Tensor:
    """y = x w^T: x [tokens, inner] in 16 bits is quantised (or comes in 8 bits from the norm before it, and y is then
    of `dtype`), w [outer, inner] is kept in 8.  scratch: a Mx8Matrix of x's size to reuse from call to call.
    The call records no autograd graph (mx8_linear_backward gives the gradients),
    so an x whose gradient autograd is to find is refused, and one with a forward-mode tangent."""
    if isinstance(x, Mx8Matrix):
        return mx8_product(x, w, dtype, out)
    if x.requires_grad and torch.is_grad_enabled():
        raise B.ZeroError(1, "mx8_linear records no autograd graph: pass x.detach() (or call it under torch.no_grad()) "
                             "and take the gradients from mx8_linear_backward")
    q = scratch.fill(x) if scratch is not None else Mx8Matrix.of(x)
    return mx8_product(q, w, x.dtype, out)


def mx8_linear_backward(dy: torch.Tensor, x: torch.Tensor, w_t: Mx8Matrix) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of y = x w^T, with the rounding of the operands passed through:
    dx = dy w and dw = dy^T x, each from operands quantised along the summed
    dimension.  w_t: w quantised along its columns (Mx8Matrix.of(w, transpose=True)).
    Both are new matrices, constants to autograd whatever dy and x require.  8192 tokens, 4096 -> 11008: 648 us, 101 of them
    the three quantisations (dy is read twice, x once)."""
    dx = mx8_product(Mx8Matrix.of(dy), w_t, dy.dtype)
    dw = mx8_product(Mx8Matrix.of(dy, True), Mx8Matrix.of(x, True), dy.dtype)
    return dx, dw

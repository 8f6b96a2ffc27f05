"""Orthogonalised momentum (the Muon optimiser) for the matrices of a partitioned model.

The matrices lie back to back in flat buffers, each at a multiple of 8
elements; :class:`MuonBuffers` owns those buffers and makes a step's calls:
the ranks' gradients into the momentum, one orthogonalisation per shape, and
the update of the fp32 master with its rounding into every rank's replica.
Everything is stream-ordered, nothing waits for the host, and a step can be
captured into a CUDA graph after it ran once.
"""

from __future__ import annotations

import math
from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import _binding as B
from .mx4 import Mx4Matrix
from .synth import torch_dtype

_ZDT = {"fp16": B.ZERO_FP16, "bf16": B.ZERO_BF16}


def aspect_scale(rows: int, cols: int) -> float:
    """sqrt(max(1, rows / cols)): the factor that keeps an update's effect alike for all shapes."""
    return math.sqrt(max(1.0, rows / cols))


class MuonBuffers:
    """The buffers of a list of matrices, [(rows, cols), ...], on N simulated ranks.

    grads and params are [N, count]; master [count] and momentum [2 * count]
    are fp32; state is the device struct of zero_muon_set_state.  The tensors
    are written in place and must not be rebound.
    """

    def __init__(self, shapes: Sequence[Tuple[int, int]], n_ranks: int, dtype: str = "bf16", device="cuda",
                 loss_scale: float = 1.0):
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        self.n, self.dtype = n_ranks, dtype
        self.offsets: List[int] = []
        at = 0
        for r, c in self.shapes:
            self.offsets.append(at)
            at += (r * c + 7) // 8 * 8
        self.count = at
        td, size = torch_dtype(dtype), max(8, at)
        self.grads = torch.zeros((n_ranks, size), dtype=td, device=device)
        self.params = torch.zeros((n_ranks, size), dtype=td, device=device)
        self.master = torch.zeros(size, device=device)
        self.momentum = torch.zeros(2 * size, device=device)
        self.update = torch.zeros(size, dtype=torch.bfloat16, device=device)
        self.ortho = torch.zeros(size, dtype=torch.bfloat16, device=device)
        self.state = torch.zeros(16, dtype=torch.int32, device=device)
        self._grad_rows = B.pointer_array(self.grads.unbind(0))
        self._param_rows = B.pointer_array(self.params.unbind(0))
        # one call per shape (and per ZERO_MAX_MATRICES matrices of it); they share the workspace
        by_shape: Dict[Tuple[int, int], List[int]] = {}
        for i, s in enumerate(self.shapes):
            if s[0] and s[1]:
                by_shape.setdefault(s, []).append(i)
        self._calls = []
        need = 0
        for (r, c), ids in by_shape.items():
            for k in range(0, len(ids), B.ZERO_MAX_MATRICES):
                part = ids[k:k + B.ZERO_MAX_MATRICES]
                need = max(need, B.zero_orthogonalize_workspace_bytes(len(part), r, c))
                self._calls.append((r, c, B.pointer_array([self.matrix(i, self.update) for i in part]),
                                    B.pointer_array([self.matrix(i, self.ortho) for i in part])))
        self.workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
        B.zero_muon_set_state(self.state, loss_scale)

    def matrix(self, i: int, flat: torch.Tensor) -> torch.Tensor:
        """Matrix i as a view of a flat row (a rank's gradients or parameters, the master, ...)."""
        r, c = self.shapes[i]
        return flat[self.offsets[i]:self.offsets[i] + r * c].view(r, c)

    def live_momentum(self, slot: int) -> torch.Tensor:
        return self.momentum[slot * self.count:(slot + 1) * self.count]

    def step(self, hyp: B.MuonHyper, steps: int = 5, coeffs=None, scale=aspect_scale, stream=None) -> None:
        """One update of all matrices from the gradients in ``grads``; scale(rows, cols) is the update's factor."""
        dt = _ZDT[self.dtype]
        B.zero_muon_momentum(dt, self.count, self._grad_rows, self.momentum, self.update, hyp, self.state, stream)
        for r, c, src, dst in self._calls:
            B.zero_orthogonalize(B.ZERO_BF16, r, c, src, dst, self.workspace, steps=steps, coeffs=coeffs,
                                 scale=float(scale(r, c)), stream=stream, state=self.state)
        B.zero_muon_apply(dt, self.count, self.ortho, self.master, self._param_rows, hyp, self.state, stream)

    def quantize(self, i: int, transpose: bool = False, rank: int = 0) -> Mx4Matrix:
        """Matrix i of a rank's replica in microscaled 4 bits, ready to multiply with.
        transpose: along its columns, as the backward pass takes it."""
        return Mx4Matrix.of(self.matrix(i, self.params[rank]), transpose)

    def status(self, stream=None) -> dict:
        """The state after the last step; raises when a kernel's bounded wait gave up (a step in whose
        orthogonalisation that happened was skipped)."""
        B.zero_matrix_status(stream)
        s = B.zero_muon_get_state(self.state, stream)
        if s["aborted"]:
            raise B.ZeroError(B.ZERO_ETIMEOUT, "a bounded wait of the last step's orthogonalisation gave up: "
                                               "the step was skipped")
        return s

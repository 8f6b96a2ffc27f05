"""Two linear layers trained on N simulated ranks with orthogonalised momentum,
their weights multiplied in microscaled 4 bits.

Every step, every rank multiplies its own tokens with the 4-bit weights
(forward and backward), and the ranks' 16-bit gradients go through
one Muon step: average, momentum, Newton-Schulz, update of the fp32 master
and of every rank's replica, from which the weights are quantised again.

    python examples/muon_mx4.py [steps]
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import zero_partitioned_mixed_gb300 as Z  # noqa: E402
from zero_partitioned_mixed_gb300.muon import MuonBuffers  # noqa: E402
from zero_partitioned_mixed_gb300.mx4 import mx4_linear, mx4_linear_backward  # noqa: E402

TOKENS, INNER, HIDDEN, OUTER, RANKS = 512, 384, 640, 200, 4


def train(steps=40, lr=0.02, seed=0):
    """The mean squared error before each step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")   # noqa: E731
    x = [rand(TOKENS, INNER).bfloat16() for _ in range(RANKS)]
    teacher = [rand(HIDDEN, INNER) / INNER ** 0.5, rand(OUTER, HIDDEN) / HIDDEN ** 0.5]
    goal = [torch.relu(b.float() @ teacher[0].t()) @ teacher[1].t() for b in x]

    buf = MuonBuffers([(HIDDEN, INNER), (OUTER, HIDDEN)], RANKS, "bf16", loss_scale=1024.0)
    for i, t in enumerate(teacher):
        buf.matrix(i, buf.master).copy_(rand(*t.shape) / t.shape[1] ** 0.5)
    buf.params.copy_(buf.master.bfloat16())
    hyper = Z.muon_hyper(lr=lr, momentum=0.9)

    losses = []
    for _ in range(steps):
        scale = buf.status()["loss_scale"]
        w1, w2, w2_t = buf.quantize(0), buf.quantize(1), buf.quantize(1, transpose=True)
        w1_t = buf.quantize(0, transpose=True)
        total = 0.0
        for r in range(RANKS):
            h = mx4_linear(x[r], w1)
            a = torch.relu(h)
            err = mx4_linear(a, w2).float() - goal[r]
            total += float((err * err).mean())
            dy = (err * (scale / TOKENS)).bfloat16()
            da, dw2 = mx4_linear_backward(dy, a, w2_t)
            _, dw1 = mx4_linear_backward(da * (h > 0), x[r], w1_t)
            buf.matrix(0, buf.grads[r]).copy_(dw1)
            buf.matrix(1, buf.grads[r]).copy_(dw2)
        losses.append(total / RANKS)
        buf.step(hyper)
    return losses


if __name__ == "__main__":
    for k, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)):
        print(f"step {k:3d}  loss {loss:.4f}")

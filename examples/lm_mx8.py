"""A small language model trained on N simulated ranks by the ZeRO stage 1 step,
its linear layers in microscaled 8 bits.

Every step, every rank runs its own tokens forward and backward: embedding,
dropout, then for each layer the norm with the residual's addition (which
writes the 8 bits that the product after it reads), two linear layers, and
the dropout of the branch inside the next norm's call.  The output layer's
weight is the embedding table.  The gradients go straight into the rank's row
of 16-bit gradients; one step averages them and updates the fp32 state.

    python examples/lm_mx8.py [steps]
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import zero_partitioned_mixed_gb300 as Z  # noqa: E402
from zero_partitioned_mixed_gb300 import layers as L  # noqa: E402
from zero_partitioned_mixed_gb300.buffers import RankBuffers  # noqa: E402
from zero_partitioned_mixed_gb300.mx8 import Mx8Matrix, mx8_linear, mx8_linear_backward  # noqa: E402

VOCAB, DIM, HIDDEN, LAYERS, TOKENS, RANKS = 203, 96, 160, 2, 120, 2
P, EPS, SEED = 0.1, 1e-5, 11


def parameters():
    """{name: shape} in the order of the flat buffers."""
    out = {"table": (VOCAB, DIM)}
    for i in range(LAYERS):
        out[f"norm{i}"], out[f"up{i}"], out[f"down{i}"] = (DIM,), (HIDDEN, DIM), (DIM, HIDDEN)
    out["norm"] = (DIM,)
    return out


class Flat:
    """The parameters' places in a flat row, each at a multiple of 8 elements."""

    def __init__(self):
        self.at, self.size = {}, 0
        for name, shape in parameters().items():
            self.at[name] = (self.size, shape)
            self.size += (torch.Size(shape).numel() + 7) // 8 * 8

    def of(self, row):
        """{name: view of the row}."""
        return {name: row[at:at + torch.Size(shape).numel()].view(shape) for name, (at, shape) in self.at.items()}


def dropouts(step):
    """One stream of numbers for each place that drops: after the embedding, and on each layer's branch."""
    return [Z.dropout_spec(P, SEED, (LAYERS + 1) * step + i) for i in range(LAYERS + 1)]


def forward(w, ids, drop):
    """(logits, what the backward pass needs) of one rank's tokens."""
    kept = {"h": [], "y": [], "up": [], "a": []}
    stream = L.dropout(L.embedding(ids, w["table"], DIM ** 0.5), drop[0])
    branch = None
    for i in range(LAYERS + 1):
        name = f"norm{i}" if i < LAYERS else "norm"
        n = (L.rms_norm(stream, w[name], EPS, bits=8) if branch is None else
             L.rms_norm(branch, w[name], EPS, residual=stream, dropout=drop[i], bits=8))
        stream = n.h
        kept["h"].append(n.h)
        kept["y"].append(n.y)
        if i < LAYERS:
            up = mx8_linear(n.q, Mx8Matrix.of(w[f"up{i}"]))
            a = torch.relu(up)
            kept["up"].append(up)
            kept["a"].append(a)
            branch = mx8_linear(a, Mx8Matrix.of(w[f"down{i}"]))
    return mx8_linear(n.q, Mx8Matrix.of(w["table"])), kept


def backward(w, g, ids, drop, kept, dlogits):
    """The gradients of all parameters into g, the views of a rank's gradient row."""
    dy, dtable = mx8_linear_backward(dlogits, kept["y"][-1], Mx8Matrix.of(w["table"], transpose=True))
    g["table"].copy_(dtable)
    dh = None
    for i in range(LAYERS, -1, -1):
        name = f"norm{i}" if i < LAYERS else "norm"
        dh, dbranch, _ = L.rms_norm_backward(dy, kept["h"][i], w[name], EPS, dh_in=dh, dropout=drop[i] if i else None,
                                             dweight=g[name])
        if i:
            da, dw = mx8_linear_backward(dbranch, kept["a"][i - 1], Mx8Matrix.of(w[f"down{i - 1}"], transpose=True))
            g[f"down{i - 1}"].copy_(dw)
            dy, dw = mx8_linear_backward(da * (kept["up"][i - 1] > 0), kept["y"][i - 1],
                                         Mx8Matrix.of(w[f"up{i - 1}"], transpose=True))
            g[f"up{i - 1}"].copy_(dw)
    # the table is also the output layer's weight: the lookup's gradient is added
    L.embedding_backward(L.dropout(dh, drop[0]), ids, g["table"], DIM ** 0.5, accumulate=True)


def loss_and_gradient(logits, target, scale):
    """Mean cross entropy, and its gradient times the loss scale in 16 bits."""
    p = torch.softmax(logits.float(), 1)
    at = torch.arange(len(target), device=p.device)
    loss = -torch.log(p[at, target]).mean()
    p[at, target] -= 1
    return loss, (p * (scale / len(target))).to(logits.dtype)


def initial(flat, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    row = torch.zeros(flat.size, device="cuda")
    for name, view in flat.of(row).items():
        if name.startswith("norm"):
            view.fill_(1.0)
        else:
            view.copy_(torch.randn(view.shape, generator=gen, device="cuda") / view.shape[1] ** 0.5)
    return row


def train(steps=30, lr=3e-3, seed=0):
    """The ranks' mean loss before each step."""
    flat = Flat()
    buf = RankBuffers(flat.size, RANKS, 1, "bf16")
    row = initial(flat, seed)
    buf.master[:flat.size] = row
    buf.params[:, :flat.size] = row.bfloat16()
    buf.set_scaler(1024.0)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    ids = [torch.randint(0, VOCAB, (TOKENS + 1,), generator=gen, device="cuda") for _ in range(RANKS)]
    losses = []
    for step in range(steps):
        drop, scale, total = dropouts(step), buf.status()["loss_scale"] if step else 1024.0, 0.0
        for r in range(RANKS):
            w, g = flat.of(buf.params[r]), flat.of(buf.grads[r])
            logits, kept = forward(w, ids[r][:-1], drop)
            loss, dlogits = loss_and_gradient(logits, ids[r][1:], scale)
            backward(w, g, ids[r][:-1], drop, kept, dlogits)
            total += float(loss)
        losses.append(total / RANKS)
        buf.step(Z.hyper(lr=lr, max_norm=1.0))
    Z.zero_matrix_status()
    return losses


if __name__ == "__main__":
    for k, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {k:3d}  loss {loss:.4f}")

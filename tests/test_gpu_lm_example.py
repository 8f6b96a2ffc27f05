"""The operators together, as examples/lm_mx8.py uses them.

Every call of a step is checked by itself, on the inputs that it gets there,
as the operators' own tests do.  The gradients of all parameters are checked
against the same model in 64 bits, which quantises where the example does
(with the library's matrices, whose values their tests hold to the
definition).  There the 16-bit roundings on the way, half a step d = 2^-8 of a
value at most, tip an 8-bit code over with a probability of d / s, s being the
codes' relative step of 2^-3 at most, and change it by s: a mean square of d s
= 2^-11, 2^-5.5 in the 2-norm.  On a gradient's longest path lie 2 layers of 2
quantised activations and the output layer's, and as many quantised gradients;
if all their errors add up, 10 * 2^-5.5, and 2^-8 for each of about 20
roundings themselves: 0.3.  (They are independent; what is seen is a quarter
of that.)  A term that is missing or wrong shows at that, and at its call."""

import importlib.util
import math
import os

import pytest
import torch

from _layer_ref import dropped, half_step, kept as kept_mask, norm64, norm_grad64, within
from _matrix_ref import rel
import zero_partitioned_mixed_gb300 as Z
from zero_partitioned_mixed_gb300.mx8 import Mx8Matrix

pytestmark = pytest.mark.gpu
LIMIT = 10 * 2.0 ** -5.5 + 20 * 2.0 ** -8
PRODUCT, GRAD, U = 2.0 ** -9, 2.0 ** -16, 2.0 ** -24     # as in the operators' own tests


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "lm_mx8.py")
    spec = importlib.util.spec_from_file_location("lm_mx8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def quantised(x, transpose=False):
    """The values that x (float64, on the CPU) has in 8 bits, along its rows or its columns; in x's shape."""
    q = Mx8Matrix.of(x.bfloat16().cuda(), transpose=transpose).values().double().cpu()
    return q.t() if transpose else q


class Linear(torch.autograd.Function):
    """y = x w^T of quantised operands; the backward products quantise theirs along what they sum over."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return quantised(x) @ quantised(w).t()

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        return quantised(dy) @ quantised(w, True), quantised(dy, True).t() @ quantised(x, True)


def reference(m, w, ids, target, masks, scale):
    """Gradients of the example's loss times `scale`, in 64 bits."""
    w = {k: v.double().cpu().requires_grad_() for k, v in w.items()}

    def drop(x, mask):
        keep, factor = mask
        return torch.where(keep, x * factor, torch.zeros((), dtype=torch.float64))

    def norm(h, weight):
        return h / torch.sqrt(h.square().mean(1, keepdim=True) + m.EPS) * weight

    h = drop(w["table"][ids] * m.DIM ** 0.5, masks[0])
    for i in range(m.LAYERS):
        a = torch.relu(Linear.apply(norm(h, w[f"norm{i}"]), w[f"up{i}"]))
        h = h + drop(Linear.apply(a, w[f"down{i}"]), masks[i + 1])
    logits = Linear.apply(norm(h, w["norm"]), w["table"])
    loss = torch.nn.functional.cross_entropy(logits, target)
    (loss * scale).backward()
    return float(loss.detach()), {k: v.grad for k, v in w.items()}


class Checked:
    """Stands in for the example's calls: makes them, and checks each one's results."""

    def __init__(self, m):
        self.m, self.calls = m, []
        self.real = {n: getattr(m.L, n) for n in ("embedding", "embedding_backward", "dropout", "rms_norm", "rms_norm_backward")}
        self.linear, self.linear_backward = m.mx8_linear, m.mx8_linear_backward
        m.L, m.mx8_linear, m.mx8_linear_backward = self, self.mx8_linear, self.mx8_linear_backward

    def mask(self, spec, like):
        return kept_mask(*like.shape, spec.p, spec.seed, spec.offset)

    def embedding(self, ids, table, scale):
        out = self.real["embedding"](ids, table, scale)
        want = (table.cpu()[ids.cpu()].float() * torch.tensor(scale, dtype=torch.float32)).bfloat16()
        assert torch.equal(out.cpu(), want)
        self.calls.append("embedding")
        return out

    def embedding_backward(self, dout, ids, dtable, scale, accumulate):
        before = dtable.double().cpu()
        out = self.real["embedding_backward"](dout, ids, dtable, scale, accumulate)
        sums = torch.zeros_like(before).index_add_(0, ids.cpu(), dout.double().cpu()) * scale
        want = sums + before if accumulate else sums
        assert within(out, want, half_step(want, out.dtype) + 2.0 ** -16 * (sums.abs() + before.abs() + 1))
        self.calls.append("embedding_backward")
        return out

    def dropout(self, x, spec):
        out = self.real["dropout"](x, spec)
        assert torch.equal(out.cpu(), dropped(x.cpu(), self.mask(spec, x)).bfloat16())
        self.calls.append("dropout")
        return out

    def rms_norm(self, x, weight, eps, residual=None, dropout=None, bits=0):
        n = self.real["rms_norm"](x, weight, eps, residual, dropout, bits)
        h = dropped(x.cpu(), self.mask(dropout, x)) if dropout is not None else x.cpu().float()
        h = (h + residual.cpu().float() if residual is not None else h).bfloat16()
        want = norm64(h, weight.cpu(), eps)[0]
        assert torch.equal(n.h.cpu(), h) and within(n.y, want, half_step(want, h.dtype) + 2.0 ** -18 * want.abs())
        far = (n.q.values().double().cpu() - want).abs()
        top = want.abs().view(len(want), -1, 32).amax(2, keepdim=True).expand(-1, -1, 32).reshape(want.shape)
        assert bool((far <= 2.0 ** -3 * want.abs() + 2.0 ** -17 * top).all())   # a saturated value is 64 of 512 off, others half a step
        self.calls.append("rms_norm")
        return n

    def rms_norm_backward(self, dy, h, weight, eps, dh_in=None, dropout=None, dweight=None):
        out = self.real["rms_norm_backward"](dy, h, weight, eps, dh_in, dropout, dweight)
        dh, dw, size, dw_size = norm_grad64(dy.cpu(), h.cpu(), weight.cpu(), eps, None if dh_in is None else dh_in.cpu())
        assert within(out[0], dh, half_step(dh, dy.dtype) + GRAD * size)
        assert within(out[2], dw, half_step(dw, dy.dtype) + 100 * U * dw_size) and out[2] is dweight
        if dropout is not None:
            keep, factor = self.mask(dropout, dy)
            dx = torch.where(keep, dh * factor, torch.zeros((), dtype=torch.float64))
            assert within(out[1], dx, half_step(dx, dy.dtype) + factor * (GRAD + U) * size)
        self.calls.append("rms_norm_backward")
        return out

    def mx8_linear(self, x, w):
        out = self.linear(x, w)
        q = x if isinstance(x, Mx8Matrix) else Mx8Matrix.of(x)
        assert rel(out, q.values().double().cpu() @ w.values().double().cpu().t()) <= PRODUCT
        self.calls.append("mx8_linear")
        return out

    def mx8_linear_backward(self, dy, x, w_t):
        dx, dw = self.linear_backward(dy, x, w_t)
        val = lambda t, tr: Mx8Matrix.of(t, transpose=tr).values().double().cpu()   # noqa: E731
        assert rel(dx, val(dy, False) @ w_t.values().double().cpu().t()) <= PRODUCT
        assert rel(dw, val(dy, True) @ val(x, True).t()) <= PRODUCT
        self.calls.append("mx8_linear_backward")
        return dx, dw


def test_gradients_of_the_example():
    m = example()
    checked = Checked(m)
    flat = m.Flat()
    row, out = m.initial(flat, 3).bfloat16(), torch.zeros(flat.size, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, m.VOCAB, (m.TOKENS + 1,), generator=torch.Generator().manual_seed(5))
    step, scale = 4, 1024.0
    drop = m.dropouts(step)
    w, g = flat.of(row), flat.of(out)
    logits, kept = m.forward(w, ids[:-1].cuda(), drop)
    loss, dlogits = m.loss_and_gradient(logits, ids[1:].cuda(), scale)
    m.backward(w, g, ids[:-1].cuda(), drop, kept, dlogits)
    Z.zero_matrix_status()
    assert {n: checked.calls.count(n) for n in set(checked.calls)} == {
        "embedding": 1, "embedding_backward": 1, "dropout": 2, "rms_norm": 3, "rms_norm_backward": 3, "mx8_linear": 5,
        "mx8_linear_backward": 5}
    masks = [kept_mask(m.TOKENS, m.DIM, m.P, m.SEED, (m.LAYERS + 1) * step + i) for i in range(m.LAYERS + 1)]
    want_loss, want = reference(m, w, ids[:-1], ids[1:], masks, scale)
    assert abs(float(loss) - want_loss) <= LIMIT * want_loss
    for name, view in g.items():
        far = float((view.double().cpu() - want[name]).norm() / want[name].norm())
        assert far <= LIMIT, f"{name}: {far}"


def test_the_example_runs():
    losses = example().train(3)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)
    assert losses == example().train(3)                 # every step repeats bit for bit

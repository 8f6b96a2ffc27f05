"""The residual stream's operators on the paths that small calls do not take.

Runs of one id in embedding gradients of up to 512 tokens, which are not
sorted: rows of one warp, of several, of all.

Sums of whole numbers below 2048 are exact in fp16 and in any order.  The
tolerances elsewhere are those of test_gpu_layers.py."""

import numpy as np
import pytest
import torch

from _layer_ref import half_step, within
from zero_partitioned_mixed_gb300 import layers as L

pytestmark = pytest.mark.gpu
TD = {"fp16": torch.float16, "bf16": torch.bfloat16}
DTYPES = ["bf16", "fp16"]
U = 2.0 ** -24
SORTED = 513     # tokens from which the gradient sorts them


def gen(seed):
    return torch.Generator().manual_seed(seed)


def whole(shape, seed, most=2):
    return torch.randint(-most, most + 1, shape, generator=gen(seed)).half()


def strided(x, offset, gap, fill=5.0):
    """x (on the GPU) as a view with a gap between its rows, and all of its storage."""
    rows, cols = x.shape
    room = torch.full((offset + rows * (cols + gap) + 32,), fill, dtype=x.dtype, device="cuda")
    view = room[offset:offset + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]
    view.copy_(x)
    return view, room


def untouched(view, room, fill=5.0):
    view.fill_(fill)
    return bool((room == fill).all())


def sums(ids, dy, vocab):
    """The rows' sums in 64 bits, on the GPU."""
    at = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    return torch.zeros((vocab + 1, dy.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, at, dy.double())[:-1]


# --------------------------------------------------- embedding, few tokens
@pytest.mark.parametrize("dim", [40, 41, 768, 1100])
def test_runs_of_few_tokens(dim):
    """Runs that one warp has all rows of, that several have and that all have: one id, some, one behind the other."""
    for tokens in (1, 9, 31, 32, 33, 34, 40, 64, 100, 255, 256, 257, 300, 511, 512, SORTED):
        for kind in range(4):
            g = gen(tokens + kind)
            ids = torch.full((tokens,), 5)
            if kind == 1:                               # half of them one id
                ids[torch.randperm(tokens, generator=g)[:tokens // 2]] = torch.randint(6, 60, (tokens // 2,), generator=g)
            elif kind == 2:                             # several ids, long runs each, and padding
                ids = torch.randint(-1, 9, (tokens,), generator=g)
            elif kind == 3:                             # runs one behind the other
                ids = torch.arange(tokens) // 33
            dy = whole((tokens, dim), tokens + kind).cuda()
            held = whole((60, dim), kind).cuda()
            for offset, gap in ((0, 0), (0, 8), (3, 5)):
                src, _ = strided(dy, offset, gap)
                for accumulate in (False, True):
                    out, room = strided(held, offset, gap)
                    L.embedding_backward(src, ids.cuda(), out, accumulate=accumulate)
                    want = sums(ids.cuda(), dy, 60)
                    assert torch.equal(out.double(), want + held.double() if accumulate else want), (tokens, kind)
                    assert untouched(out, room)


@pytest.mark.parametrize("dtype", DTYPES)
def test_sums_of_few_tokens_are_fp32_and_repeat(dtype):
    tokens, dim, vocab = 500, 300, 12
    ids = torch.randint(-1, 4, (tokens,), generator=gen(1)).cuda()
    dy = (torch.randn((tokens, dim), generator=gen(2)) * 0.1).to(TD[dtype]).cuda()
    want, size = (sums(ids, t, vocab).cpu() * np.float32(1.7) for t in (dy, dy.abs()))
    count = torch.bincount(ids[ids >= 0], minlength=vocab).double().cpu().unsqueeze(1)
    out = torch.full((vocab, dim), float("nan"), dtype=TD[dtype], device="cuda")
    L.embedding_backward(dy, ids, out, 1.7)
    assert within(out, want, torch.where(size > 0, half_step(want, TD[dtype]) + (count + 1) * U * size, 0.0))
    for _ in range(5):
        again = torch.full_like(out, 3.0)
        L.embedding_backward(dy, ids.int(), again, 1.7)
        assert torch.equal(again, out)

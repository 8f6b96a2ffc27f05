"""The residual stream's operators on the paths that small calls do not take.

Embedding gradients of more than 512 tokens (sorted) over every digit count of
the sort, rows at every alignment, tables past 32 bits, captured; runs of one
id that begin and end at every place of their pieces of 8 tokens; and of up to
512 tokens, which are not sorted: rows of one warp, of several, of all.  The
norm's backward pass with several rows for each row of threads, so that its
ring of copies, its sums and its share of the weight's gradient go round.

Sums of whole numbers below 2048 are exact in fp16 and in any order.  The
tolerances elsewhere are those of test_gpu_layers.py, the one of the weight's
gradient with the blocks that there are: the workspace has a row of fp32 for
each."""

import numpy as np
import pytest
import torch

from _layer_ref import half_step, kept, norm_grad64, within
import zero_partitioned_mixed_gb300 as Z
from zero_partitioned_mixed_gb300 import layers as L

pytestmark = pytest.mark.gpu
TD = {"fp16": torch.float16, "bf16": torch.bfloat16}
DTYPES = ["bf16", "fp16"]
U, GRAD = 2.0 ** -24, 2.0 ** -16
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


# -------------------------------------------------- embedding, many tokens
@pytest.mark.parametrize("tokens", [600, 5000, 20011])
@pytest.mark.parametrize("vocab", [2 ** 16 - 1, 2 ** 16, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 5, 2 ** 31 - 1, 2 ** 31])
def test_sorted_ids_of_every_digit_count(vocab, tokens):
    ids = torch.randint(0, vocab, (tokens,), generator=gen(tokens))
    ids[:40] = vocab - 1 - torch.arange(40) % 7
    ids[40:80] = torch.arange(40) % 5
    ids[80:130] = torch.tensor([-1, vocab, 2 ** 40, -2 ** 50, 2 ** 32]).repeat(10)       # padding
    ids[130:200] = (1 << torch.arange(70) % 31) % vocab                                  # one bit each
    ids = ids[torch.randperm(tokens, generator=gen(1))].cuda()
    dy = whole((tokens, 1), tokens).cuda()
    out = torch.full((vocab, 1), 7.0, dtype=torch.float16, device="cuda")
    L.embedding_backward(dy, ids, out)
    inside = (ids >= 0) & (ids < vocab)
    rows, back = torch.unique(ids[inside], return_inverse=True)
    want = torch.zeros(len(rows), dtype=torch.float64, device="cuda").index_add_(0, back, dy[inside, 0].double())
    assert torch.equal(out[rows, 0].double(), want)
    out[rows] = 0.0
    assert not any(bool(part.any()) for part in out.split(1 << 28))


def test_sorted_gradient_of_a_table_past_32_bits():
    vocab, dim, tokens = 1_100_003, 4000, 700           # 4.4e9 elements
    ids = (vocab - 1 - torch.randint(0, 90, (tokens,), generator=gen(1))).cuda()
    ids[::7] = 3
    dy = whole((tokens, dim), 2).cuda()
    out = torch.full((vocab, dim), 7.0, dtype=torch.float16, device="cuda")
    for accumulate in (False, True):
        L.embedding_backward(dy, ids, out, accumulate=accumulate)
        rows = torch.unique(ids)
        at = torch.searchsorted(rows, ids)
        want = sums(at, dy, len(rows)) * (1 + accumulate)
        assert torch.equal(out[rows].double(), want)
    out[rows] = 0.0
    assert not any(bool(part.any()) for part in out.split(100_000))


WIDTHS = list(range(1, 42)) + [63, 64, 65, 121, 127, 128, 129] + list(range(247, 266)) + [300, 503, 511, 512, 513, 520, 777, 1017, 1025]


@pytest.mark.parametrize("offset", range(8))
def test_sorted_gradient_of_rows_of_every_alignment_and_width(offset):
    vocab, tokens = 97, SORTED + 88
    for cols in WIDTHS:
        gap = (cols * 5 + offset) % 8
        ids = torch.randint(-2, vocab + 2, (tokens,), generator=gen(cols)).cuda()
        ids[offset * 20:offset * 20 + 150] = 31         # a run that the join adds up by a block
        dy, _ = strided(whole((tokens, cols), cols).cuda(), offset, gap)
        held = whole((vocab, cols), cols + 1).cuda()
        want = sums(ids, dy, vocab)
        for accumulate in (False, True):
            out, room = strided(held, (3 * offset + 1) % 8, gap)
            L.embedding_backward(dy, ids, out, accumulate=accumulate)
            assert torch.equal(out.double(), want + held.double() if accumulate else want), cols
            assert untouched(out, room), cols


@pytest.mark.parametrize("pieces", [1, 2, 8, 9, 10, 31, 32, 33, 34, 65, 97])
@pytest.mark.parametrize("dim", [40, 41])
def test_runs_at_every_place_of_their_pieces(dim, pieces):
    """A run that covers so many pieces of 8 sorted tokens, from each place of its first to three of its last; other runs
    before and behind it, and padding up to the sorted form."""
    for begin in range(8):
        for end in (1, 5, 8):
            length = 8 * pieces - begin - (8 - end)
            if length < 1:
                continue
            for behind in (0, 3):
                ids = torch.cat((torch.arange(begin), torch.full((length,), 20), 21 + torch.arange(behind)))
                ids = torch.cat((ids, torch.full((max(0, SORTED - len(ids)),), -1)))
                perm = torch.randperm(len(ids), generator=gen(pieces))
                ids = ids[perm].cuda()
                dy = whole((len(ids), dim), length).cuda()
                out = torch.full((30, dim), 9.0, dtype=torch.float16, device="cuda")
                L.embedding_backward(dy, ids, out)
                assert torch.equal(out.double(), sums(ids, dy, 30)), (begin, end, behind)


def test_captured_sorted_gradients():
    """Two graphs that share a workspace and run in order; the replays sort the ids that are there then."""
    vocab, dim, tokens = 3000, 264, 4100
    ids, dy = torch.zeros(tokens, dtype=torch.int64, device="cuda"), torch.zeros((tokens, dim), dtype=torch.float16, device="cuda")
    room = torch.empty(Z.zero_embedding_backward_workspace_bytes(vocab, dim, tokens), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((vocab, dim), dtype=torch.float16, device="cuda") for _ in range(2)]
    L.embedding_backward(dy, ids, outs[0], workspace=room)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in outs]
    for graph, out, scale in zip(graphs, outs, (1.0, 2.0)):
        with torch.cuda.graph(graph):
            L.embedding_backward(dy, ids, out, scale, workspace=room)
            L.embedding_backward(dy, ids, out, scale, True, room)
    for k in range(4):
        new = torch.randint(-5, vocab + 5, (tokens,), generator=gen(k))
        new[k * 100:k * 100 + 90 * k] = 77 + k
        ids.copy_(new)
        dy.copy_(whole((tokens, dim), k, 1))
        for _ in range(3):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        want = sums(ids, dy, vocab)
        assert torch.equal(outs[0].double(), 2 * want) and torch.equal(outs[1].double(), 4 * want)


# ------------------------------------------------------ norm, backward pass
def mask(rows, cols, p, seed, stream):
    """_layer_ref.kept for many rows: the generator in numpy's 64-bit whole numbers."""
    low, groups = np.uint64(0xFFFFFFFF), (cols + 7) // 8
    n = np.arange(rows * groups, dtype=np.uint64)
    c = [n & low, n >> np.uint64(32), np.full_like(n, stream & 0xFFFFFFFF), np.full_like(n, stream >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [k[0] + 0x9E3779B9 & 0xFFFFFFFF, k[1] + 0xBB67AE85 & 0xFFFFFFFF]
    halves = np.stack([w >> np.uint64(16 * h) & np.uint64(0xFFFF) for w in c for h in (0, 1)], 1).reshape(rows, groups * 8)
    drop = round(p * 65536)
    return torch.from_numpy(halves[:, :cols] >= drop), float(np.float32(65536 / (65536 - drop)))


#: Rows, columns, and how many rows a block has at a time: every row of threads takes three to five rows.
LOOPS = [(8000, 96, 8), (8000, 99, 8), (7400, 776, 8), (7400, 777, 8), (4000, 520, 2), (4000, 523, 2), (2000, 2184, 1),
         (2000, 2187, 1), (1000, 4096, 1), (1000, 5003, 1), (1000, 9000, 1), (1000, 9001, 1), (950, 16384, 1), (950, 16001, 1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,slots", LOOPS)
def test_norm_backward_of_several_rows_a_thread(rows, cols, slots, dtype):
    g = gen(rows + cols)
    h = torch.randn((rows, cols), generator=g) * torch.exp(0.5 * torch.randn((rows, 1), generator=g))
    if dtype == "bf16":   # some rows' squares leave fp32, on either side
        h *= torch.tensor([1.0, 1.0, 2.0 ** 70, 1.0, 2.0 ** -70, 1.0, 2.0 ** 100]).repeat(rows // 7 + 1)[:rows, None]
    h, w = h.to(TD[dtype]), torch.randn(cols, generator=g).to(TD[dtype])
    dy, d = ((0.1 * torch.randn((rows, cols), generator=g)).to(TD[dtype]) for _ in range(2))
    blocks = Z.zero_rms_norm_backward_workspace_bytes(rows, cols) // (4 * 8 * ((cols + 7) // 8))
    assert rows > 3 * blocks * slots
    keep, factor = mask(rows, cols, 0.1, 3, 4)
    small = kept(3, cols, 0.1, 3, 4)
    assert torch.equal(keep[:3], small[0]) and factor == small[1]
    dh, dw, size, dw_size = norm_grad64(dy, h, w, 1e-5, d)
    dx = torch.where(keep, dh * factor, torch.zeros((), dtype=torch.float64))
    # additions to dw: a thread's rows, a block's rows of threads, a warp's shares, 32 warps; and r's roundings
    adds = -(-rows // (blocks * slots)) + slots + -(-blocks // 32) + 32 + 36
    spec = Z.dropout_spec(0.1, 3, 4)
    for offset, gap in ((0, 0), (3, 5)):
        hs, ys, ds = (strided(t.cuda(), offset, gap)[0] for t in (h, dy, d))
        got = L.rms_norm_backward(ys, hs, w.cuda(), 1e-5, ds, spec)
        assert within(got[0], dh, half_step(dh, TD[dtype]) + GRAD * size)
        assert within(got[1], dx, half_step(dx, TD[dtype]) + factor * (GRAD + U) * size)
        assert within(got[2], dw, half_step(dw, TD[dtype]) + adds * U * dw_size)
        for _ in range(3):
            again = L.rms_norm_backward(ys, hs, w.cuda(), 1e-5, ds, spec)
            assert all(torch.equal(a, b) for a, b in zip(got, again))
        # in place: the stream's gradient where the incoming one was, the branch's where the output's was
        ld, room = cols + gap, torch.empty(Z.zero_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        dweight = torch.empty_like(w, device="cuda")
        Z.zero_rms_norm_backward({"fp16": 0, "bf16": 1}[dtype], rows, cols, ys, hs, w.cuda(), 1e-5, ds, room, ds, ys, dweight, spec,
                                 ld, ld, ld, ld, ld)
        assert torch.equal(ds, got[0]) and torch.equal(ys, got[1]) and torch.equal(dweight, got[2])


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

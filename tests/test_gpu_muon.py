"""Orthogonalised momentum on the GPU: the momentum and apply streams bit for
bit against fp32 arithmetic on the CPU, the Newton-Schulz orthogonalisation
against 64 bits, whole steps, refusals.

Tolerance of the orthogonalisation (2-norm of the error over that of the
result).  The result is rounded to bf16: 2^-9 at most, 1.7e-3 over many
values.  The intermediate matrices are rounded to fp16 (2^-12 at most); a
64-bit model of the same rounding points gives 1.0e-3 to 2.3e-3 in all from
sides of 16 up, and up to 1.3e-2 below, where a matrix has few values to
average over and may be badly conditioned.  The bounds are those with a
factor of about two: 5e-3 from 16 up, 2.5e-2 below."""

import numpy as np
import pytest
import torch

from _matrix_ref import DEFAULT, gradient, newton_schulz, rel
import zero_partitioned_mixed_gb300 as Z
from zero_partitioned_mixed_gb300.muon import MuonBuffers, aspect_scale

pytestmark = pytest.mark.gpu
TD = {"fp16": torch.float16, "bf16": torch.bfloat16}
ZD = {"fp16": Z.ZERO_FP16, "bf16": Z.ZERO_BF16}


def bound(rows, cols):
    return 5e-3 if min(rows, cols) >= 16 else 2.5e-2


def workspace(batch, rows, cols):
    return torch.full((Z.zero_orthogonalize_workspace_bytes(batch, rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")


def ortho(src, **kw):
    """src [batch, rows, cols] on the GPU -> bf16."""
    b, r, c = src.shape
    dst = torch.full((b, r, c), 7.0, dtype=torch.bfloat16, device="cuda")
    Z.zero_orthogonalize(ZD["bf16" if src.dtype == torch.bfloat16 else "fp16"], r, c, list(src.unbind(0)),
                         list(dst.unbind(0)), workspace(b, r, c), **kw)
    Z.zero_matrix_status()
    return dst


SIZES = [(1, 1), (1, 40), (40, 1), (3, 5), (8, 8), (16, 16), (31, 33), (64, 64), (65, 63), (96, 160), (127, 128),
         (128, 129), (129, 127), (200, 2049), (2049, 200), (256, 256), (255, 511), (384, 640), (700, 300), (513, 1030),
         (1030, 513), (1024, 1024), (128, 512), (128, 513), (513, 128), (20, 4096), (4096, 100), (128, 4097), (4100, 77),
         (1, 3000), (129, 4096), (257, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_orthogonalize_matches_64_bits(rows, cols, dtype):
    g = gradient(rows, cols, rows * 31 + cols, batch=2).to(TD[dtype])
    got = ortho(g.cuda())
    for i in range(2):
        assert rel(got[i], newton_schulz(g[i].double())) <= bound(rows, cols)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 5, 4097), (1, 100, 8192), (1, 8191, 128), (20, 37, 5001), (3, 6000, 16),
                                             (1, 64, 8193), (1, 8193, 33), (40, 128, 2600), (8, 2049, 90), (9, 2176, 128)])
def test_long_thin_matrices(batch, rows, cols, dtype):
    """Lengths around what a cluster of 8 and one of 16 blocks holds, more matrices than such clusters fit at once."""
    g = gradient(rows, cols, rows * 31 + cols, batch=batch).to(TD[dtype])
    got = ortho(g.cuda())
    for i in sorted({0, batch // 2, batch - 1}):
        x = g[i].double()
        want = newton_schulz(x.t()).t() if rows > cols else newton_schulz(x)   # the shorter side's Gram matrix
        assert rel(got[i], want) <= bound(rows, cols)
    assert torch.equal(got, ortho(g.cuda()))


@pytest.mark.parametrize("rows,cols", [(90, 1537), (1537, 90), (33, 512), (511, 128), (5001, 24), (24, 8190), (7, 3)])
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (5, 8), (7, 2), (8, 8)])
def test_thin_matrices_at_any_alignment(rows, cols, offset, pad):
    """The result does not depend on where rows start, and nothing beside them is written."""
    ld = cols + pad
    g = gradient(rows, cols, rows + 7 * cols).to(torch.bfloat16).cuda()
    want = ortho(g)[0]
    src = torch.full((offset + rows * ld + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    dst = torch.full((offset + rows * ld + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    view = (rows, cols), (ld, 1), offset
    src.as_strided(*view).copy_(g[0])
    Z.zero_orthogonalize(Z.ZERO_BF16, rows, cols, [src[offset:]], [dst[offset:]], workspace(1, rows, cols), ld_src=ld,
                         ld_dst=ld)
    assert torch.equal(dst.as_strided(*view), want)
    dst.as_strided(*view).fill_(7.0)
    assert bool((dst == 7.0).all())


@pytest.mark.parametrize("batch", [1, 5, 128])
def test_batches_are_independent(batch):
    g = gradient(72, 104, batch, batch=batch).bfloat16().cuda()
    got = ortho(g)
    for i in {0, batch // 2, batch - 1}:
        assert torch.equal(got[i:i + 1], ortho(g[i:i + 1].clone()))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("rows,cols", [(48, 200), (200, 48)])
def test_steps_coefficients_and_scale(steps, rows, cols):
    g = gradient(rows, cols, steps).bfloat16()
    coeffs = [DEFAULT, (3.0, -3.2, 1.2), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
    coeffs = (coeffs * 2)[:steps]
    got = ortho(g.cuda(), steps=steps, coeffs=coeffs, scale=-0.37)
    assert rel(got[0], newton_schulz(g[0].double(), steps, coeffs, -0.37)) <= 5e-3


@pytest.mark.parametrize("dtype,factor", [("bf16", 2.0 ** 100), ("bf16", 2.0 ** 67), ("bf16", 2.0 ** -100),
                                          ("bf16", 2.0 ** -60), ("fp16", 2.0 ** 13)])
def test_scale_of_the_input_does_not_matter(dtype, factor):
    g = (1e3 * gradient(80, 112, 5)).to(TD[dtype]).cuda()
    far = (g.double() * factor).to(TD[dtype])
    assert torch.equal(far.double(), g.double() * factor)
    assert torch.equal(ortho(far), ortho(g))


def test_zero_infinity_and_nan_stay_in_their_matrix():
    g = gradient(70, 90, 3, batch=5).bfloat16().cuda()
    clean = ortho(g.clone())
    g[1] = 0
    g[2, 69, 89] = float("inf")
    g[3, 0, 0] = float("nan")
    got = ortho(g)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[4], clean[4])
    assert not got[1].any()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()


def test_rank_one_and_zero_rows():
    u, v = torch.randn(60, 1, generator=torch.Generator().manual_seed(1)), torch.randn(1, 200, generator=torch.Generator().manual_seed(2))
    g = (u @ v)[None].bfloat16()
    g[0, 7] = 0
    got = ortho(g.cuda())
    # one large singular value beside rounding noise far below it; the zero row stays zero
    assert not got[0, 7].any()
    assert rel(got[0], newton_schulz(g[0].double())) <= 2.5e-2


@pytest.mark.parametrize("offset,ld", [(0, 104), (1, 97), (3, 131), (8, 97)])
def test_strides_alignment_and_guard_bands(offset, ld):
    rows, cols, batch = 65, 97, 3
    g = gradient(rows, cols, 11, batch=batch).bfloat16().cuda()
    want = ortho(g)
    room = rows * ld + 64
    src = torch.full((batch, room), float("nan"), dtype=torch.bfloat16, device="cuda")
    dst = torch.full((batch, room), 5.0, dtype=torch.bfloat16, device="cuda")
    view = lambda t, i: t[i, offset:offset + rows * ld].view(rows, ld)[:, :cols]   # noqa: E731
    for i in range(batch):
        view(src, i).copy_(g[i])
    Z.zero_orthogonalize(Z.ZERO_BF16, rows, cols, [view(src, i) for i in range(batch)],
                         [view(dst, i) for i in range(batch)], workspace(batch, rows, cols), ld_src=ld, ld_dst=ld)
    for i in range(batch):
        assert torch.equal(view(dst, i), want[i])
        view(dst, i).fill_(5.0)
    assert bool((dst == 5.0).all())     # nothing beside the matrices was written


def test_workspace_is_not_exceeded_and_repeats_are_bitwise():
    rows, cols, batch = 130, 258, 3
    g = gradient(rows, cols, 9, batch=batch).bfloat16().cuda()
    n = Z.zero_orthogonalize_workspace_bytes(batch, rows, cols)
    ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = []
    for _ in range(3):
        dst = torch.empty_like(g)
        Z.zero_orthogonalize(Z.ZERO_BF16, rows, cols, list(g), list(dst), ws[:n])
        out.append(dst)
    assert bool((ws[n:] == 0xA5).all())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_in_place_other_stream_and_graph():
    g = gradient(300, 180, 4, batch=2).bfloat16().cuda()
    want = ortho(g)
    ws = workspace(2, 300, 180)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mine = g.clone()
    with torch.cuda.stream(s):
        Z.zero_orthogonalize(Z.ZERO_BF16, 300, 180, list(mine), list(mine), ws)
    s.synchronize()
    assert torch.equal(mine, want)
    graph, src, dst = torch.cuda.CUDAGraph(), torch.zeros_like(g), torch.zeros_like(g)
    with torch.cuda.graph(graph):
        Z.zero_orthogonalize(Z.ZERO_BF16, 300, 180, list(src), list(dst), ws)
    src.copy_(g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dst, want)


def test_calls_in_a_row_on_shared_scratch():
    ws = workspace(4, 520, 520)
    cases = [gradient(r, c, r, batch=2).bfloat16().cuda() for r, c in ((64, 500), (520, 520), (500, 64), (17, 33))]
    want = [ortho(g) for g in cases]
    got = [torch.empty_like(g) for g in cases]
    for g, o in list(zip(cases, got)) * 2:
        Z.zero_orthogonalize(Z.ZERO_BF16, g.shape[1], g.shape[2], list(g), list(o), ws)
    for o, w in zip(got, want):
        assert torch.equal(o, w)


# ----------------------------------------------------------- the two streams
def sum_ranks(grads, scale):
    s = np.zeros(grads.shape[1], np.float32)
    for r in grads:
        s = s + r.float().numpy()
    return s / np.float32(np.float32(len(grads)) * np.float32(scale))


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ranks,count", [(1, 1), (2, 7), (3, 8), (4, 4099), (8, 100_003), (9, 65_536), (64, 5001)])
@pytest.mark.parametrize("nesterov,scale", [(True, 1024.0), (False, 1000.0)])
def test_momentum_is_bit_exact(ranks, count, dtype, nesterov, scale):
    gen = torch.Generator().manual_seed(ranks * count)
    pad = (count + 7) // 8 * 8
    grads = torch.full((ranks, pad + 8), 3.0, dtype=TD[dtype])
    grads[:, :count] = torch.randn((ranks, count), generator=gen).to(TD[dtype])
    m = torch.zeros(2 * pad + 8)
    m[:count] = torch.randn(count, generator=gen)
    m[count:] = 9.0
    state = torch.zeros(16, dtype=torch.int32, device="cuda")
    Z.zero_muon_set_state(state, scale)
    dm, du = m.cuda(), torch.full((pad + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
    Z.zero_muon_momentum(ZD[dtype], count, [r for r in grads.cuda()], dm, du, Z.muon_hyper(momentum=0.9, nesterov=nesterov), state)
    g = sum_ranks(grads[:, :count], scale)
    mu = np.float32(0.9)
    new = mu * m[:count].numpy() + g
    upd = g + mu * new if nesterov else new
    assert np.array_equal(dm[pad:pad + count].cpu().numpy().view(np.uint32), new.view(np.uint32))
    assert torch.equal(dm[:pad].cpu(), m[:pad]) and bool((dm[pad + count:] == 9.0).all())
    assert torch.equal(du[:count].cpu(), bf16_bits(upd)) and bool((du[count:] == 9.0).all())
    s = Z.zero_muon_get_state(state)
    assert s["pending"] == 0 and s["slot"] == 0 and s["steps_applied"] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ranks,count,shift", [(1, 1, 0), (3, 13, 0), (8, 100_003, 0), (5, 4096, 4), (64, 777, 4)])
def test_apply_is_bit_exact(ranks, count, shift, dtype):
    gen = torch.Generator().manual_seed(count)
    w = torch.full((count + 8 + shift,), 9.0)     # shift 4: 16-byte but not 32-byte aligned state
    w[shift:shift + count] = torch.randn(count, generator=gen)
    o = torch.randn(count, generator=gen).bfloat16()
    pad = (count + 7) // 8 * 8
    params = torch.full((ranks, pad + 8), 9.0, dtype=TD[dtype], device="cuda")
    state = torch.zeros(16, dtype=torch.int32, device="cuda")
    Z.zero_muon_set_state(state, 4.0, 11, 1)
    dw = w.cuda()
    Z.zero_muon_apply(ZD[dtype], count, o.cuda(), dw[shift:], list(params), Z.muon_hyper(lr=0.02, weight_decay=0.1), state)
    lr, decay = np.float32(0.02), np.float32(1.0 - float(np.float32(0.02)) * float(np.float32(0.1)))
    want = w[shift:shift + count].numpy() * decay - lr * o.float().numpy()
    got = dw.cpu().numpy()
    assert np.array_equal(got[shift:shift + count].view(np.uint32), want.view(np.uint32))
    assert (got[shift + count:] == 9.0).all() and (got[:shift] == 9.0).all()
    p16 = torch.from_numpy(want).to(TD[dtype])
    for r in range(ranks):
        assert torch.equal(params[r, :count].cpu(), p16) and bool((params[r, count:] == 9.0).all())
    s = Z.zero_muon_get_state(state)
    assert (s["steps_applied"], s["slot"], s["applied"], s["overflow"], s["loss_scale"]) == (12, 0, 1, 0, 4.0)


def test_empty_calls():
    state = torch.zeros(16, dtype=torch.int32, device="cuda")
    Z.zero_muon_set_state(state)
    Z.zero_muon_momentum(Z.ZERO_BF16, 0, [None], None, None, Z.muon_hyper(), state)
    Z.zero_muon_apply(Z.ZERO_BF16, 0, None, None, [None], Z.muon_hyper(), state)
    assert Z.zero_muon_get_state(state)["steps_applied"] == 1
    Z.zero_orthogonalize(Z.ZERO_BF16, 0, 5, [], [], None)
    Z.zero_orthogonalize(Z.ZERO_BF16, 5, 0, [None], [None], None)


# --------------------------------------------------------------- whole steps
SHAPES = [(48, 80), (80, 48), (33, 65), (48, 80), (1, 70)]


def plain_step(shapes, grads, masters, moms, scale, lr, decay, mu):
    """One step in 64 bits, from the same 16-bit gradients; the update rounded to bf16 as the definition has it."""
    out_w, out_m = [], []
    for i, (r, c) in enumerate(shapes):
        g = sum(grads[k][i].double() for k in range(len(grads))) / (len(grads) * scale)
        m = mu * moms[i] + g
        u = (g + mu * m).float().bfloat16().double()
        out_w.append((1 - lr * decay) * masters[i] - lr * newton_schulz(u, scale=aspect_scale(r, c)))
        out_m.append(m)
    return out_w, out_m


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_steps_follow_the_plain_form_and_skip_overflow(dtype):
    ranks, lr, decay, mu, scale = 3, 0.02, 0.1, 0.95, 256.0
    buf = MuonBuffers(SHAPES, ranks, dtype, loss_scale=scale)
    hyp = Z.muon_hyper(lr=lr, momentum=mu, weight_decay=decay)
    gen = torch.Generator().manual_seed(8)
    masters, moms = [], []
    for i, (r, c) in enumerate(SHAPES):
        w = 0.02 * torch.randn((r, c), generator=gen)
        buf.matrix(i, buf.master).copy_(w)
        masters.append(w.double())
        moms.append(torch.zeros(r, c, dtype=torch.float64))
    for step in range(4):
        grads = [[(scale * gradient(r, c, 100 * step + 10 * k + i)[0]).to(TD[dtype]) for i, (r, c) in enumerate(SHAPES)]
                 for k in range(ranks)]
        for k in range(ranks):
            for i in range(len(SHAPES)):
                buf.matrix(i, buf.grads[k]).copy_(grads[k][i])
        if step == 2:
            before = [t.clone() for t in (buf.master, buf.params)]
            buf.matrix(3, buf.grads[1])[5, 6] = float("inf")
        buf.step(hyp)
        s = buf.status()
        if step == 2:
            assert (s["overflow"], s["applied"], s["steps_skipped"], s["loss_scale"]) == (1, 0, 1, scale / 2)
            assert torch.equal(buf.master, before[0]) and torch.equal(buf.params, before[1])
            scale /= 2
            continue
        assert s["applied"] == 1 and s["overflow"] == 0
        masters, moms = plain_step(SHAPES, grads, masters, moms, scale, lr, decay, mu)
        for i, (r, c) in enumerate(SHAPES):
            got = buf.matrix(i, buf.master).double().cpu()
            # each step adds lr * bound of the orthogonalised update's norm, at most
            size = lr * aspect_scale(r, c) * 1.25 * min(r, c) ** 0.5
            assert float((got - masters[i]).norm()) <= (step + 1) * size * bound(r, c)
            assert rel(buf.matrix(i, buf.live_momentum(s["slot"])), moms[i]) <= 1e-5
            for k in range(ranks):
                assert torch.equal(buf.matrix(i, buf.params[k]), buf.matrix(i, buf.master).to(TD[dtype]))
    assert Z.zero_muon_get_state(buf.state)["steps_applied"] == 3


def test_a_captured_step_replays_like_calls():
    hyp = Z.muon_hyper(lr=0.01)
    bufs = [MuonBuffers(SHAPES, 2, "bf16") for _ in range(2)]
    for b in bufs:
        b.step(hyp)                       # on zero gradients: loads the kernels
        assert not b.master.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bufs[1].step(hyp)
    for step in range(3):
        for b in bufs:
            for k in range(2):
                for i, (r, c) in enumerate(SHAPES):
                    b.matrix(i, b.grads[k]).copy_(gradient(r, c, step * 50 + k * 7 + i)[0])
        bufs[0].step(hyp)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0].master, bufs[1].master) and torch.equal(bufs[0].params, bufs[1].params)
        assert bufs[0].status() == bufs[1].status()
    assert bufs[1].master.any()


def test_the_example_trains():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "muon_mx4.py")
    spec = importlib.util.spec_from_file_location("muon_mx4_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=25)
    assert all(np.isfinite(losses))
    # 25 steps of an update whose size is the learning rate reach well below half of the start
    assert losses[-1] < 0.5 * losses[0] and min(losses) == min(losses[5:])
    assert losses == mod.train(steps=25)     # every kernel of the path gives the same bits again


# ------------------------------------------------- offsets past 32 bits
def test_a_batch_whose_offsets_pass_32_bits():
    side, batch = 5800, 128          # 4.3e9 elements
    src = torch.empty((batch, side, side), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    one = torch.randn((side, side), generator=gen, device="cuda")
    for i in range(batch):
        src[i] = one.roll(37 * i, 1) * (1.0 + i)
    ws = torch.empty(Z.zero_orthogonalize_workspace_bytes(batch, side, side), dtype=torch.uint8, device="cuda")
    Z.zero_orthogonalize(Z.ZERO_BF16, side, side, list(src.unbind(0)), list(src.unbind(0)), ws, steps=2)   # in place
    for i in (0, 127):
        mine = (one.roll(37 * i, 1) * (1.0 + i)).bfloat16()
        Z.zero_orthogonalize(Z.ZERO_BF16, side, side, [mine], [mine], ws, steps=2)
        assert torch.equal(mine, src[i])
    Z.zero_matrix_status()


def test_a_flat_region_whose_offsets_pass_32_bits():
    count, tail = (1 << 32) + 1003, 5000
    grads = torch.zeros((2, count + 5), dtype=torch.bfloat16, device="cuda")      # rows of whole eights
    momentum = torch.zeros(2 * (count + 5), device="cuda")
    update = torch.zeros(count + 5, dtype=torch.bfloat16, device="cuda")
    master, params = torch.zeros(count + 5, device="cuda"), torch.zeros((1, count + 5), dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(16, dtype=torch.int32, device="cuda")
    Z.zero_muon_set_state(state)
    gen = torch.Generator(device="cuda").manual_seed(2)
    grads[:, count - tail:count] = torch.randn((2, tail), generator=gen, device="cuda").bfloat16()
    hyp = Z.muon_hyper(lr=0.5, momentum=0.5)
    Z.zero_muon_momentum(Z.ZERO_BF16, count, list(grads.unbind(0)), momentum, update, hyp, state)
    Z.zero_muon_apply(Z.ZERO_BF16, count, update, master, list(params.unbind(0)), hyp, state)
    g = (grads[0, count - tail:count].float() + grads[1, count - tail:count].float()) * 0.5
    u = (g + 0.5 * g).bfloat16()
    assert torch.equal(momentum[2 * (count + 5) - 5 - tail:-5], g)
    assert torch.equal(update[count - tail:count], u)
    assert torch.equal(master[count - tail:count], -0.5 * u.float())
    assert torch.equal(params[0, count - tail:count], (-0.5 * u.float()).bfloat16())
    assert not update[:count - tail].any() and not master[count:].any()


# ------------------------------------------------------------------ refusals
def test_refusals():
    t = torch.zeros(4096, device="cuda")
    h = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(16, dtype=torch.int32, device="cuda")
    ws = workspace(1, 16, 16)
    hyp = Z.muon_hyper()

    def refused(text, fn, *a, **kw):
        with pytest.raises(Z.ZeroError) as e:
            fn(*a, **kw)
        assert e.value.code == 1 and text in str(e.value), str(e.value)

    mom, app, ns = Z.zero_muon_momentum, Z.zero_muon_apply, Z.zero_orthogonalize
    refused("dtype", mom, 5, 8, [h], t, h, hyp, state)
    refused("n_ranks", mom, 0, 8, [h] * 65, t, h, hyp, state)
    refused("grads[r]", mom, 0, 8, [h, None], t, h, hyp, state)
    refused("grads[r]", mom, 0, 8, [h[1:]], t, h, hyp, state)
    refused("momentum", mom, 0, 8, [h], t[1:], h, hyp, state)
    refused("update", mom, 0, 8, [h], t, h[1:], hyp, state)
    refused("momentum must lie", mom, 0, 8, [h], t, h, Z.muon_hyper(momentum=1.0), state)
    refused("finite", mom, 0, 8, [h], t, h, Z.muon_hyper(lr=float("nan")), state)
    refused("state", mom, 0, 8, [h], t, h, hyp, None)
    refused("ortho", app, 0, 8, None, t, [h], hyp, state)
    refused("master", app, 0, 8, h, None, [h], hyp, state)
    refused("params[r]", app, 0, 8, h, t, [h, h[3:]], hyp, state)
    refused("loss_scale", Z.zero_muon_set_state, state, 0.0)
    refused("slot", Z.zero_muon_set_state, state, 1.0, 0, 2)
    refused("dtype", ns, 2, 16, 16, [h], [h], ws)
    refused("batch", ns, 0, 16, 16, [h] * 129, [h] * 129, ws)
    refused("steps", ns, 0, 16, 16, [h], [h], ws, steps=0)
    refused("steps", ns, 0, 16, 16, [h], [h], ws, steps=33)
    refused("scale", ns, 0, 16, 16, [h], [h], ws, scale=float("inf"))
    refused("coeffs", ns, 0, 16, 16, [h], [h], ws, coeffs=(1.0, float("nan"), 0.0))
    refused("coeffs", ns, 0, 16, 16, [h], [h], ws, coeffs=[(1.0, 0.0, 0.0)] * 3)
    refused("ld_src", ns, 0, 16, 16, [h], [h], ws, ld_src=15)
    refused("src[i]", ns, 0, 16, 16, [None], [h], ws)
    refused("dst[i]", ns, 0, 16, 16, [h], [None], ws)
    refused("same length", ns, 0, 16, 16, [h], [], ws)
    refused("workspace", ns, 0, 16, 16, [h], [h], None)
    refused("are needed", ns, 0, 16, 16, [h], [h], ws[:-1])
    refused("ZERO_MAX_SIDE", ns, 0, (1 << 18) + 1, 16, [h], [h], ws)
    assert Z.zero_orthogonalize_workspace_bytes(1, (1 << 18) + 1, 16) == 0
    torch.cuda.synchronize()


# ------------------------------------------- an orthogonalisation that could not finish
@pytest.mark.parametrize("pending,scale", [(2, 512.0), (3, 256.0), (1, 256.0)])
def test_what_a_wait_that_gave_up_left_is_not_applied(pending, scale):
    """The word that such a wait sets (2) and a non-finite gradient's (1), written by the host."""
    buf = MuonBuffers(SHAPES, 2, "bf16", loss_scale=512.0)
    hyp = Z.muon_hyper(lr=0.1)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in (buf.grads, buf.params, buf.master):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    buf.step(hyp)
    first = buf.status()
    assert first["applied"] == 1 and first["aborted"] == 0
    before = [t.clone() for t in (buf.master, buf.params, buf.live_momentum(first["slot"]))]
    Z.zero_muon_momentum(Z.ZERO_BF16, buf.count, list(buf.grads), buf.momentum, buf.update, hyp, buf.state)
    buf.state[2] |= pending
    buf.ortho.fill_(7.0)
    Z.zero_muon_apply(Z.ZERO_BF16, buf.count, buf.ortho, buf.master, list(buf.params), hyp, buf.state)
    s = Z.zero_muon_get_state(buf.state)
    assert torch.equal(buf.master, before[0]) and torch.equal(buf.params, before[1])
    assert s["slot"] == first["slot"] and torch.equal(buf.live_momentum(s["slot"]), before[2])
    assert (s["overflow"], s["applied"], s["steps_applied"], s["steps_skipped"]) == (1, 0, 1, 1)
    assert (s["aborted"], s["loss_scale"], s["pending"]) == (pending >> 1, scale, 0)
    if s["aborted"]:
        with pytest.raises(Z.ZeroError) as e:
            buf.status()
        assert e.value.code == 4
    buf.step(hyp)
    s = buf.status()
    assert (s["applied"], s["aborted"], s["steps_applied"]) == (1, 0, 2)
    assert not torch.equal(buf.master, before[0])


HELD = [(1, 64, 96), (1, 96, 64), (1, 100, 2000), (2, 1500, 40), (1, 60, 6000), (3, 300, 180), (2, 180, 700)]


@pytest.mark.parametrize("batch,rows,cols", HELD)
@pytest.mark.parametrize("stage", [0, 2])
def test_a_wait_that_runs_out_ends_the_call_and_is_reported(batch, rows, cols, stage):
    """Both kernels, in one block and in clusters: block 0 stops feeding the tensor cores on purpose."""
    g = gradient(rows, cols, rows + cols, batch=batch).bfloat16().cuda()
    want = ortho(g)
    ws = workspace(batch, rows, cols)
    room = torch.full((batch, rows * cols + 512), 7.0, dtype=torch.bfloat16, device="cuda")
    dst = [t[256:256 + rows * cols].view(rows, cols) for t in room]
    Z._binding.zero_debug_hold_matrix(stage)
    Z.zero_orthogonalize(Z.ZERO_BF16, rows, cols, list(g), dst, ws)
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_matrix_status()
    assert e.value.code == 4 and "zero_orthogonalize" in str(e.value)
    for _ in range(2):
        Z.zero_orthogonalize(Z.ZERO_BF16, rows, cols, list(g), dst, ws)
    Z.zero_matrix_status()
    for d, w in zip(dst, want):
        assert torch.equal(d, w)
        d.fill_(7.0)
    assert bool((room == 7.0).all())


@pytest.mark.parametrize("shape", [(48, 80), (90, 1100), (300, 180)])
def test_a_step_whose_orthogonalisation_gave_up_is_skipped(shape):
    hyp = Z.muon_hyper(lr=0.05, weight_decay=0.1)
    bufs = [MuonBuffers([shape, (33, 65)], 2, "fp16", loss_scale=128.0) for _ in range(2)]
    gen = torch.Generator().manual_seed(5)
    w = [0.02 * torch.randn(s, generator=gen) for s in bufs[0].shapes]
    for b in bufs:
        for i in range(2):
            b.matrix(i, b.master).copy_(w[i])
        b.params.copy_(b.master.half())

    def gradients(step):
        for b in bufs:
            for k in range(2):
                for i, (r, c) in enumerate(b.shapes):
                    b.matrix(i, b.grads[k]).copy_(128 * gradient(r, c, 40 * step + 10 * k + i)[0])

    gradients(0)
    for b in bufs:
        b.step(hyp)
    a, b = bufs
    a.status()
    before = [t.clone() for t in (b.master, b.params)]
    Z._binding.zero_debug_hold_matrix(1)      # the first matrix of the next step
    b.step(hyp)
    s = Z.zero_muon_get_state(b.state)
    assert (s["applied"], s["overflow"], s["aborted"], s["steps_applied"], s["loss_scale"]) == (0, 1, 1, 1, 128.0)
    assert torch.equal(b.master, before[0]) and torch.equal(b.params, before[1])
    for _ in range(2):                        # the device's word, then the step's own
        with pytest.raises(Z.ZeroError) as e:
            b.status()
        assert e.value.code == 4
    gradients(1)
    for c in bufs:                            # as if the skipped step had not been
        c.step(hyp)
    assert torch.equal(a.master, b.master) and torch.equal(a.params, b.params)
    sa, sb = a.status(), b.status()
    assert torch.equal(a.live_momentum(sa["slot"]), b.live_momentum(sb["slot"]))
    assert sb["steps_skipped"] == 1 and sa["steps_applied"] == sb["steps_applied"] == 2


# ------------------- shorter sides above 128: the products through global memory, at what the tests above hold at small sizes
# Bounds as above; the 64-bit model of the rounding points gives 1.7e-3 to 1.9e-3 for the step counts here and 9.8e-3
# for the matrices of rank one.
@pytest.mark.parametrize("batch", [1, 5, 128])
def test_large_batches_are_independent(batch):
    g = gradient(172, 204, batch, batch=batch).bfloat16().cuda()
    got = ortho(g)
    for i in {0, batch // 2, batch - 1}:
        assert torch.equal(got[i:i + 1], ortho(g[i:i + 1].clone()))


@pytest.mark.parametrize("steps", [1, 2, 3, 8, 32])
@pytest.mark.parametrize("rows,cols", [(150, 290), (290, 150), (260, 520)])
def test_large_steps_coefficients_and_scale(steps, rows, cols):
    g = gradient(rows, cols, steps).bfloat16()
    coeffs = [DEFAULT, (3.0, -3.2, 1.2), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
    coeffs = (coeffs * 8)[:steps]
    got = ortho(g.cuda(), steps=steps, coeffs=coeffs, scale=-0.37)
    assert rel(got[0], newton_schulz(g[0].double(), steps, coeffs, -0.37)) <= 5e-3


@pytest.mark.parametrize("dtype,factor", [("bf16", 2.0 ** 100), ("bf16", 2.0 ** 67), ("bf16", 2.0 ** -100),
                                          ("bf16", 2.0 ** -60), ("fp16", 2.0 ** 13)])
def test_scale_of_a_large_input_does_not_matter(dtype, factor):
    g = (1e3 * gradient(180, 212, 5)).to(TD[dtype]).cuda()
    far = (g.double() * factor).to(TD[dtype])
    assert torch.equal(far.double(), g.double() * factor)
    assert torch.equal(ortho(far), ortho(g))


@pytest.mark.parametrize("rows,cols", [(170, 290), (290, 170)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_zero_infinity_and_nan_stay_in_their_large_matrix(rows, cols, dtype):
    g = (100 * gradient(rows, cols, 3, batch=6)).to(TD[dtype]).cuda()
    clean = ortho(g.clone())
    g[1] = 0
    g[2, rows - 1, cols - 1] = float("inf")
    g[3, 0, 0] = float("nan")
    g[4, rows // 2, 7] = -float("inf")
    got = ortho(g)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[5], clean[5])
    assert not got[1].any()
    assert all(torch.isnan(got[i]).all() for i in (2, 3, 4))


@pytest.mark.parametrize("rows,cols", [(160, 300), (300, 160)])
def test_large_rank_one_and_zero_rows(rows, cols):
    u, v = (torch.randn(*s, generator=torch.Generator().manual_seed(k)) for s, k in (((rows, 1), 1), ((1, cols), 2)))
    g = (u @ v)[None].bfloat16()
    g[0, 7] = 0
    got = ortho(g.cuda())
    assert not got[0, 7].any()
    assert rel(got[0], newton_schulz(g[0].double())) <= 2.5e-2


@pytest.mark.parametrize("rows,cols", [(165, 297), (297, 165)])
@pytest.mark.parametrize("offset,pad", [(0, 7), (1, 0), (3, 34), (8, 3), (0, 23)])
def test_large_strides_alignment_and_guard_bands(rows, cols, offset, pad):
    ld, batch = cols + pad, 3
    g = gradient(rows, cols, 11, batch=batch).bfloat16().cuda()
    want = ortho(g)
    room = offset + rows * ld + 64
    src = torch.full((batch, room), float("nan"), dtype=torch.bfloat16, device="cuda")
    dst = torch.full((batch, room), 5.0, dtype=torch.bfloat16, device="cuda")
    view = lambda t, i: t[i, offset:offset + rows * ld].view(rows, ld)[:, :cols]   # noqa: E731
    for i in range(batch):
        view(src, i).copy_(g[i])
    Z.zero_orthogonalize(Z.ZERO_BF16, rows, cols, [view(src, i) for i in range(batch)],
                         [view(dst, i) for i in range(batch)], workspace(batch, rows, cols), ld_src=ld, ld_dst=ld)
    for i in range(batch):
        assert torch.equal(view(dst, i), want[i])
        view(dst, i).fill_(5.0)
    assert bool((dst == 5.0).all())

"""The residual stream's operators on the GPU against 64-bit references.

Where the fp32 arithmetic is exact or a single rounding, results are compared
bit for bit (dropout, lookup, sums of whole numbers, norms whose factor is a
power of two).  Elsewhere a value may be off by half a step of its type
(half_step) and by the fp32 roundings before it, u = 2^-24 each:
  norm      the sum of squares passes 32 additions in a thread, 5 in a warp and
            16 warps at most, the mean, the root and the two factors 6 more
            roundings: 59 u on the sum, half of it on its root, 36 u < 2^-18
  backward  the same for r, three times in its cubes, and the sum of g h: 2^-16
            of the magnitudes that are added and cancel
  dweight   rows / blocks additions in a thread, 8 warps, 10 shares in a
            warp, 32 warps, and r's 36 u
  embedding n additions for a token that comes n times, and the factor"""

import numpy as np
import pytest
import torch

from _layer_ref import DECODE, ENCODE, dropped, half_step, kept, norm64, norm_grad64, within
import zero_partitioned_mixed_gb300 as Z
from zero_partitioned_mixed_gb300 import layers as L
from zero_partitioned_mixed_gb300.mx4 import Mx4Matrix
from zero_partitioned_mixed_gb300.mx8 import Mx8Matrix

pytestmark = pytest.mark.gpu
TD = {"fp16": torch.float16, "bf16": torch.bfloat16}
DTYPES = ["bf16", "fp16"]
U = 2.0 ** -24
NORM, GRAD = 2.0 ** -18, 2.0 ** -16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def matrix(rows, cols, dtype, seed, size=1.0):
    g = gen(seed)
    return (size * torch.randn((rows, cols), generator=g) * torch.exp(0.5 * torch.randn((rows, 1), generator=g))).to(TD[dtype])


def strided(x, offset, gap, fill=5.0):
    """x on the GPU as a view with a gap between its rows, and all of its storage."""
    rows, cols = x.shape
    room = torch.full((offset + rows * (cols + gap) + 32,), fill, dtype=x.dtype, device="cuda")
    view = room[offset:offset + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]
    view.copy_(x)
    return view, room


def untouched(view, room, fill=5.0):
    view.fill_(fill)
    return bool((room == fill).all())


LAYOUTS = [(0, 0), (0, 8), (1, 0), (3, 5), (8, 1)]


# ----------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,p", [(1, 1, 0.5), (1, 7, 0.9), (3, 8, 0.1), (5, 9, 0.25), (33, 129, 0.1), (70, 264, 0.5),
                                         (2, 4100, 0.3)])
def test_dropout_is_exact(rows, cols, p, dtype):
    x = matrix(rows, cols, dtype, rows + cols)
    mask = kept(rows, cols, p, 2 ** 40 + 17, 3)
    spec = Z.dropout_spec(p, 2 ** 40 + 17, 3)
    want = dropped(x, mask).to(TD[dtype])
    for offset, gap in LAYOUTS:
        src, _ = strided(x, offset, gap)
        dst, room = strided(torch.zeros_like(x), (offset + 2) % 9, gap)
        assert torch.equal(L.dropout(src, spec).cpu(), want)
        L.dropout(src, spec, out=dst)
        assert torch.equal(dst.cpu(), want) and untouched(dst, room)
        L.dropout(src, spec, out=src)                   # in place
        assert torch.equal(src.cpu(), want)
    assert torch.equal(L.dropout(x.cuda(), Z.dropout_spec(0.0, 1)).cpu(), x)
    # the backward pass is the same call
    dy = matrix(rows, cols, dtype, 9)
    assert torch.equal(L.dropout(dy.cuda(), spec).cpu(), dropped(dy, mask).to(TD[dtype]))


def test_dropout_of_many_dimensions_is_that_of_its_rows():
    x = matrix(6, 72, "bf16", 1)
    spec = Z.dropout_spec(0.3, 5)
    assert torch.equal(L.dropout(x.view(2, 3, 72).cuda(), spec).view(6, 72), L.dropout(x.cuda(), spec))
    assert torch.equal(L.dropout(x[0].cuda(), spec), L.dropout(x.cuda(), spec)[0])


@pytest.mark.parametrize("p", [0.02, 0.1, 0.5, 0.97])
def test_dropout_drops_its_share(p):
    n = 1 << 22
    kept_share = float((L.dropout(torch.ones(n, dtype=torch.bfloat16, device="cuda"), Z.dropout_spec(p, 77)) != 0).double().mean())
    # six standard deviations of a share of n independent draws
    assert abs(kept_share - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -17
    a, b = (L.dropout(torch.ones(n, dtype=torch.bfloat16, device="cuda"), Z.dropout_spec(p, *k)) != 0 for k in ((77, 1), (78, 0)))
    both = float((a & b).double().mean())               # other streams and seeds: independent
    assert abs(both - (1 - p) ** 2) < 6 * ((1 - p) ** 2 * (1 - (1 - p) ** 2) / n) ** 0.5 + 2.0 ** -15


def test_dropped_values_are_zero_whatever_they_were():
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.0] * 50, dtype=torch.bfloat16).view(1, 200)
    keep, factor = kept(1, 200, 0.5, 4, 0)
    got = L.dropout(x.cuda(), Z.dropout_spec(0.5, 4)).cpu()
    assert not got[~keep].any() and torch.equal(torch.isnan(got), torch.isnan(x) & keep)
    assert torch.equal(got[keep & torch.isfinite(x)], torch.full((int((keep & torch.isfinite(x)).sum()),), 6.0, dtype=torch.bfloat16))


def test_dropout_past_32_bits():
    rows, cols = 1_100_000, 4096                        # 4.5e9 elements, 5.6e8 groups
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    spec = Z.dropout_spec(0.5, 9)
    L.dropout(x, spec, out=x)
    keep, _ = kept(2, cols, 0.5, 9, 0, first_row=rows - 2)
    assert torch.equal(x[-2:].cpu() != 0, keep)
    del x
    rows, cols, ld = 3, 9, 1 << 31                      # rows far apart
    room = torch.ones(2 * ld + 16, dtype=torch.bfloat16, device="cuda")
    view = room.as_strided((rows, cols), (ld, 1))
    got = L.dropout(view, spec)
    assert torch.equal(got.cpu() != 0, kept(rows, cols, 0.5, 9, 0)[0])


def test_dropout_of_more_values_than_an_odd_row_may_have():
    # 2^34 values and more, without gaps, from 2 bytes behind a boundary: its rows are short
    rows, cols = 2 ** 22 + 3, 4096
    room = torch.ones(rows * cols + 1, dtype=torch.bfloat16, device="cuda")
    x = room[1:].view(rows, cols)
    L.dropout(x, Z.dropout_spec(0.5, 9), out=x)
    for first in (0, 2 ** 21 - 1, rows - 2):
        assert torch.equal(x[first:first + 2].cpu() != 0, kept(2, cols, 0.5, 9, 0, first_row=first)[0])
    assert float(room[0]) == 1.0


# --------------------------------------------------- rows at any alignment
WIDTHS = list(range(1, 42)) + [63, 64, 65, 121, 127, 128, 129] + list(range(247, 266)) + [300, 503, 511, 512, 513, 520, 777, 1017, 1025]


@pytest.mark.parametrize("offset", range(8))
def test_rows_of_every_alignment_and_width(offset):
    """Copies through every way of reading and writing a row: its first and last pieces, the ends of warps, and
    nothing beside it."""
    spec = Z.dropout_spec(0.0, 1)
    for cols in WIDTHS:
        gap = (cols * 5 + offset) % 8                   # rows of one matrix at several alignments
        x = torch.randint(-2 ** 15, 2 ** 15, (5, cols), generator=gen(cols), dtype=torch.int16)
        x = torch.where((x & 0x7C00) == 0x7C00, x & 0x3FFF, x).view(torch.float16)       # any number
        src, src_room = strided(x, offset, gap)
        dst, room = strided(torch.zeros_like(x), (3 * offset + 1) % 8, gap)
        L.dropout(src, spec, out=dst)
        assert torch.equal(dst.cpu().view(torch.int16), x.view(torch.int16)) and untouched(dst, room), cols
        ids = torch.tensor([4, 0, 3, -1, 1], device="cuda")
        L.embedding(ids, src, out=dst)
        want = x[ids.cpu().clamp(min=0)].clone()
        want[3] = 0
        assert torch.equal(dst.cpu().view(torch.int16), want.view(torch.int16)) and untouched(dst, room), cols
        back = torch.tensor([2, 0, 4, 1, 3], device="cuda")       # each row from one token
        L.embedding_backward(src, back, dst)
        assert torch.equal(dst[back].cpu(), x) and untouched(dst, room), cols
        assert untouched(src, src_room)


@pytest.mark.parametrize("rows", [3, 310, 1220])
def test_norm_rows_of_every_alignment_and_width(rows):
    # (threads have one, two and four groups of a row)
    w = torch.ones(2100, dtype=torch.float16, device="cuda")
    for k, cols in enumerate(WIDTHS + [1400, 2049]):
        offset, gap = k % 8, (k * 3) % 8
        x = torch.randint(-9, 10, (rows, cols), generator=gen(cols)).half()
        src, _ = strided(x, offset, gap)
        h, h_room = strided(torch.zeros_like(x), (offset * 5 + 2) % 8, gap)
        y, y_room = strided(torch.zeros_like(x), (offset + 3) % 8, gap)
        Z.zero_rms_norm(0, rows, cols, src, w, 1e-5, src, h, y, ld_x=cols + gap, ld_residual=cols + gap, ld_h=cols + gap,
                        ld_out=cols + gap)
        assert torch.equal(h.cpu(), 2 * x), cols
        want, _ = norm64(2 * x, w[:cols].cpu(), 1e-5)
        assert within(y, want, half_step(want, torch.float16) + NORM * want.abs()), cols
        assert untouched(h, h_room) and untouched(y, y_room), cols
        if rows > 400:
            continue
        dy = torch.randint(-3, 4, (rows, cols), generator=gen(cols + 1)).half()
        g, _ = strided(dy, (offset + 6) % 8, gap)
        dh, dh_room = strided(torch.zeros_like(x), (offset * 3 + 1) % 8, gap)
        dw = torch.full((cols + 16,), 5.0, dtype=torch.float16, device="cuda")
        room = torch.empty(Z.zero_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        ld = cols + gap
        Z.zero_rms_norm_backward(0, rows, cols, g, src, w, 1e-5, dh, room, dweight16=dw[8:], ld_dy=ld, ld_h=ld, ld_dh=ld)
        want, want_w, size, w_size = norm_grad64(dy, x, w[:cols].cpu(), 1e-5)
        assert within(dh, want, half_step(want, torch.float16) + GRAD * size), cols
        adds = rows / 100 + 8 + 10 + 32 + 36
        assert within(dw[8:8 + cols], want_w, half_step(want_w, torch.float16) + adds * U * w_size), cols
        assert untouched(dh, dh_room) and bool((dw[:8] == 5).all()) and bool((dw[8 + cols:] == 5).all()), cols


# -------------------------------------------------------------------- norm
SIZES = [(1, 1), (1, 8), (2, 31), (3, 256), (9, 257), (5, 768), (131, 100), (4, 1003), (3, 1024), (2, 1025), (3, 4096),
         (2, 8200), (2, 16384), (257, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("residual,p", [(False, 0.0), (True, 0.0), (True, 0.1), (False, 0.3)])
def test_norm(rows, cols, residual, p, dtype):
    x, r, w = matrix(rows, cols, dtype, 1), matrix(rows, cols, dtype, 2), matrix(1, cols, dtype, 3)[0]
    spec = Z.dropout_spec(p, 11, 5) if p else None
    v = dropped(x, kept(rows, cols, p, 11, 5)) if p else x.float()
    h = (v + r.float() if residual else v).to(TD[dtype])          # fp32, each operation rounded once
    for offset, gap in LAYOUTS[:1] + LAYOUTS[2:4]:
        xs, rs = strided(x, offset, gap)[0], strided(r, offset, gap)[0]
        got = L.rms_norm(xs, w.cuda(), 1e-5, rs if residual else None, spec)
        assert torch.equal(got.h.cpu(), h)
        want, _ = norm64(h, w, 1e-5)
        assert within(got.y, want, half_step(want, TD[dtype]) + NORM * want.abs())
    assert got.q is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,gap", LAYOUTS)
def test_norm_keeps_its_bounds(offset, gap, dtype):
    rows, cols = 37, 203
    x, r, w = (strided(matrix(rows, cols, dtype, k), offset, gap) for k in (1, 2, 3))
    ws = torch.full((cols + 16,), float("nan"), dtype=TD[dtype], device="cuda")
    ws[offset:offset + cols] = w[0][0]
    h, out = (strided(torch.zeros(rows, cols, dtype=TD[dtype]), (offset + k) % 9, gap) for k in (1, 4))
    for bits, kind in ((4, Mx4Matrix), (8, Mx8Matrix)):
        nc, ns = kind._codes_bytes(rows, cols), kind._scales_bytes(rows, cols)
        codes, scales = (torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda") for n in (nc, ns))
        Z.zero_rms_norm({"fp16": 0, "bf16": 1}[dtype], rows, cols, x[0], ws[offset:], 1e-5, r[0], h[0], out[0], bits, codes, scales,
                        ld_x=cols + gap, ld_residual=cols + gap, ld_h=cols + gap, ld_out=cols + gap)
        assert bool((codes[nc:] == 0xA5).all()) and bool((scales[ns:] == 0xA5).all())
        plain = L.rms_norm(x[0].contiguous(), ws[offset:offset + cols].clone(), 1e-5, r[0].contiguous(), bits=bits)
        assert torch.equal(plain.h, h[0]) and torch.equal(plain.y, out[0])
        assert torch.equal(plain.q.codes[:nc], codes[:nc]) and torch.equal(plain.q.scales[:ns], scales[:ns])
    assert untouched(*h) and untouched(*out)


def test_norm_in_place():
    x, r, w = (matrix(50, 333, "bf16", k).cuda() for k in (1, 2, 3))
    want = L.rms_norm(x, w[0].clone(), residual=r)
    a, b = x.clone(), r.clone()
    Z.zero_rms_norm(1, 50, 333, a, w[0].clone(), 1e-5, b, h16=b, out16=a)
    assert torch.equal(b, want.h) and torch.equal(a, want.y)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 33), (3, 96), (2, 1024), (130, 129), (5, 1500), (2, 4096), (1, 16300)])
def test_norm_codes_are_exact_where_its_factor_is(rows, cols, bits):
    # every value of a row has one magnitude, a power of two: with eps 0 the norm is the sign, and y = +- weight
    g = gen(cols)
    sign = torch.randint(0, 2, (rows, cols), generator=g) * 2.0 - 1
    x = (sign * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g).float())).bfloat16()
    w = (torch.randn(cols, generator=g) * torch.exp2(torch.randint(-9, 9, (cols,), generator=g).float())).bfloat16()
    got = L.rms_norm(x.cuda(), w.cuda(), 0.0, bits=bits)
    y = sign.double() * w.double()
    assert torch.equal(got.y.double().cpu(), y)
    q = (Mx4Matrix if bits == 4 else Mx8Matrix).of(got.y)         # the quantiser's own tests hold it to the definition
    nc, ns = q._codes_bytes(rows, cols), q._scales_bytes(rows, cols)
    assert torch.equal(got.q.codes[:nc], q.codes[:nc]) and torch.equal(got.q.scales[:ns], q.scales[:ns])
    codes, scales = ENCODE[bits](y.numpy())
    assert np.array_equal(got.q.values().double().cpu().numpy(), DECODE[bits](codes, scales, cols))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_codes_round_once(bits, dtype):
    # the fp32 result is within 2^-18 of y, and rounding is monotone: a code lies between those of y's neighbours
    x, w = matrix(40, 500, dtype, 1), matrix(1, 500, dtype, 2)[0]
    y = norm64(x, w, 1e-5)[0]
    got = L.rms_norm(x.cuda(), w.cuda(), bits=bits, wide=False)
    assert got.y is None
    v = got.q.values(torch.float16).double().cpu().numpy().copy()
    low, high = (DECODE[bits](*ENCODE[bits]((y * (1 + s * NORM)).numpy()), 500) for s in (-1, 1))
    low, high = np.minimum(low, high), np.maximum(low, high)
    low, high = (torch.from_numpy(b).half().double().numpy() for b in (low, high))
    assert ((low <= v) & (v <= high)).all()
    assert (low == high).mean() > 0.99                  # the bounds say something


def test_special_rows_stay_alone():
    w = torch.rand(300, generator=gen(1)).bfloat16() + 0.5
    x = matrix(12, 300, "bf16", 2)
    clean = L.rms_norm(x.cuda(), w.cuda(), bits=8)
    x[2], x[5, 299], x[7, 0], x[9, 31] = 0.0, float("nan"), float("inf"), 3e38
    got = L.rms_norm(x.cuda(), w.cuda(), bits=8)
    rest = [i for i in range(12) if i not in (2, 5, 7, 9)]
    assert torch.equal(got.y[rest], clean.y[rest]) and torch.equal(got.q.values()[rest], clean.q.values()[rest])
    assert not got.y[2].any() and not got.q.values()[2].any()     # zeros: eps keeps the factor finite
    assert torch.isnan(got.y[5]).all() and torch.isnan(got.q.values()[5]).all()
    assert torch.isnan(got.y[7, 0]) and not got.y[7, 1:].any()    # infinity times 0
    assert torch.isnan(got.q.values()[7, :32]).all() and not got.q.values()[7, 32:].any()
    big = norm64(x[9:10], w, 1e-5)[0]                             # the square leaves fp32, and the others are next to nothing
    assert within(got.y[9:10], big, half_step(big, torch.bfloat16) + NORM * big.abs())
    zero = L.rms_norm(torch.zeros(3, 300, dtype=torch.bfloat16, device="cuda"), w.cuda(), 0.0, bits=8)
    assert torch.isnan(zero.y).all() and torch.isnan(zero.q.values()).all()   # 0 / 0


OUTSIDE = [2.0 ** e for e in (0, 66, -70, 56, 100, -100, 120, -30, 60, -80)]


@pytest.mark.parametrize("rows,cols", [(10, 1), (10, 8), (10, 300), (11, 1003), (10, 4096), (10, 16384), (310, 260), (1300, 520), (1300, 301)])
def test_norm_of_rows_whose_squares_leave_fp32(rows, cols):
    h, dy, w = matrix(rows, cols, "bf16", 1), matrix(rows, cols, "bf16", 2, 0.1), matrix(1, cols, "bf16", 3)[0]
    h = (h.float() * torch.tensor(OUTSIDE).repeat(rows // 10 + 1)[:rows, None]).bfloat16()
    for offset, gap in LAYOUTS[:1] + LAYOUTS[3:4]:
        hs, ys = strided(h, offset, gap)[0], strided(dy, offset, gap)[0]
        for eps in (0.0, 1e-5):
            want, _ = norm64(h, w, eps)
            got = L.rms_norm(hs, w.cuda(), eps, bits=8)
            assert within(got.y, want, half_step(want, torch.bfloat16) + NORM * want.abs())
            code = L.rms_norm(hs, w.cuda(), eps, bits=8, wide=False).q
            assert torch.equal(code.codes, got.q.codes) and torch.equal(code.scales, got.q.scales)
            tops = want.abs().amax(1)                   # the scale words follow the values
            assert within(got.q.values().double().cpu().abs().amax(1), tops, tops / 8)
            check_backward(L.rms_norm_backward(ys, hs, w.cuda(), eps), dy, h, w, eps, None, None, "bf16", rows)


# ---------------------------------------------------------- norm, backward
def check_backward(got, dy, h, w, eps, dh_in, mask, dtype, rows, exact_dx=True):
    dh, dw, size, dw_size = norm_grad64(dy, h, w, eps, dh_in)
    assert within(got[0], dh, half_step(dh, TD[dtype]) + GRAD * size)
    adds = rows / 100 + 8 + 10 + 32 + 36                # at least 100 blocks, or one row a thread
    assert within(got[2], dw, half_step(dw, TD[dtype]) + adds * U * dw_size)
    if mask is not None:
        keep, factor = mask
        want = torch.where(keep, dh * factor, torch.zeros((), dtype=torch.float64))
        assert within(got[1], want, half_step(want, TD[dtype]) + factor * (GRAD + U) * size)
        assert not got[1].cpu()[~keep].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES + [(700, 96), (400, 1100)])
@pytest.mark.parametrize("stream,p", [(True, 0.0), (True, 0.1), (False, 0.0), (False, 0.3)])
def test_norm_backward(rows, cols, stream, p, dtype):
    h, dy, d, w = (matrix(rows, cols, dtype, k, s) for k, s in ((1, 1.0), (2, 0.1), (3, 0.1), (4, 1.0)))
    w = w[0]
    spec, mask = (Z.dropout_spec(p, 3, 4), kept(rows, cols, p, 3, 4)) if p else (None, None)
    for offset, gap in LAYOUTS[:1] + LAYOUTS[3:4]:      # (rows at other alignments are added up in another order)
        hs, ys, ds = (strided(t, offset, gap)[0] for t in (h, dy, d))
        outs = [L.rms_norm_backward(ys, hs, w.cuda(), 1e-5, ds if stream else None, spec) for _ in range(2)]
        check_backward(outs[0], dy, h, w, 1e-5, d if stream else None, mask, dtype, rows)
        assert (outs[0][1] is outs[0][0]) == (spec is None)
        assert all(torch.equal(a, b) for a, b in zip(*outs))        # it repeats bit for bit


@pytest.mark.parametrize("offset,gap", LAYOUTS)
def test_norm_backward_keeps_its_bounds(offset, gap):
    rows, cols = 37, 203
    h, dy, d = (strided(matrix(rows, cols, "bf16", k), offset, gap) for k in (1, 2, 3))
    w = matrix(1, cols, "bf16", 4)[0].cuda()
    dh, dx = (strided(torch.zeros(rows, cols).bfloat16(), (offset + k) % 9, gap) for k in (1, 4))
    dw = strided(torch.zeros(1, cols).bfloat16(), offset, 0)
    need = Z.zero_rms_norm_backward_workspace_bytes(rows, cols)
    room = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    spec, ld = Z.dropout_spec(0.2, 1), cols + gap
    Z.zero_rms_norm_backward(1, rows, cols, dy[0], h[0], w, 1e-5, dh[0], room[:need], d[0], dx[0], dw[0], spec, ld, ld, ld, ld, ld)
    want = L.rms_norm_backward(dy[0].contiguous(), h[0].contiguous(), w, 1e-5, d[0].contiguous(), spec)
    assert all(torch.equal(a, b) for a, b in zip((dh[0], dx[0], dw[0][0]), want))
    assert untouched(*dh) and untouched(*dx) and untouched(*dw) and bool((room[need:] == 0xA5).all())
    # without the weight's gradient no workspace is needed, and dh may take the place of what it is made of
    for place in (dy, d):
        a, b = dy[0].clone(), d[0].clone()
        a, b = strided(a.cpu(), offset, gap)[0], strided(b.cpu(), offset, gap)[0]
        Z.zero_rms_norm_backward(1, rows, cols, a, h[0], w, 1e-5, a if place is dy else b, None, b, None, None, None, ld, ld, ld, ld)
        assert torch.equal(a if place is dy else b, want[0])


def test_norm_backward_against_differences():
    # the loss sum(y * c) in 64 bits: central differences of the reference's own forward pass, to 1e-6
    h, c, w = matrix(4, 50, "bf16", 1), matrix(4, 50, "bf16", 2), matrix(1, 50, "bf16", 3)[0]
    dh, _, dw = L.rms_norm_backward(c.cuda(), h.cuda(), w.cuda(), 1e-3)
    loss = lambda h, w: float((norm64(h, w, 1e-3)[0] * c.double()).sum())   # noqa: E731
    e = 1e-4
    for i, j in ((0, 0), (1, 49), (3, 20)):
        a, b = h.double().clone(), h.double().clone()
        a[i, j] += e
        b[i, j] -= e
        slope = (loss(a, w) - loss(b, w)) / (2 * e)
        size = norm_grad64(c, h, w, 1e-3)[2][i, j]
        assert abs(float(dh[i, j]) - slope) <= 2.0 ** -8 * abs(slope) + GRAD * float(size) + 1e-6
    for j in (0, 31, 49):
        a, b = w.double().clone(), w.double().clone()
        a[j] += e
        b[j] -= e
        slope = (loss(h, a) - loss(h, b)) / (2 * e)
        assert abs(float(dw[j]) - slope) <= 2.0 ** -8 * abs(slope) + 1e-6


# --------------------------------------------------------------- embedding
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,dim,tokens", [(1, 1, 1), (5, 8, 3), (40, 33, 70), (300, 256, 1), (1000, 257, 130), (50, 1024, 9),
                                              (70, 5000, 5)])
def test_embedding_is_exact(vocab, dim, tokens, dtype):
    table = matrix(vocab, dim, dtype, 1)
    ids = torch.randint(0, vocab, (tokens,), generator=gen(2))
    ids[::3] = torch.tensor([-1, vocab, 2 ** 40, -2 ** 40])[torch.arange(len(ids[::3])) % 4]      # padding
    inside = (ids >= 0) & (ids < vocab)
    rows = torch.where(inside.unsqueeze(1), table[ids.clamp(0, vocab - 1)].float(), torch.zeros(()))
    for scale in (1.0, 27.712812921102035):
        want = (rows * torch.tensor(scale, dtype=torch.float32)).to(TD[dtype])
        for offset, gap in LAYOUTS:
            t = strided(table, offset, gap)[0]
            out, room = strided(torch.zeros(tokens, dim, dtype=TD[dtype]), (offset + 3) % 9, gap)
            assert torch.equal(L.embedding(ids.cuda(), t, scale).cpu(), want)
            short = torch.where(inside, ids, -1).int()
            L.embedding(short.cuda(), t, scale, out=out)
            assert torch.equal(out.cpu(), want) and untouched(out, room)


def sums64(ids, dy, vocab):
    out, size, count = (torch.zeros((vocab + 1, dy.shape[1]), dtype=torch.float64) for _ in range(3))
    at = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    out.index_add_(0, at, dy.double())
    size.index_add_(0, at, dy.double().abs())
    count.index_add_(0, at, torch.ones_like(dy, dtype=torch.float64))
    return out[:-1], size[:-1], count[:-1]


GRADS = [(1, 1, 1), (2, 5, 40), (7, 64, 17), (255, 96, 500), (256, 33, 1000), (300, 257, 16), (70000, 8, 3000), (50, 300, 9000),
         (1000, 40, 20001), (2 ** 24 + 5, 1, 100), (9, 2100, 33), (4000, 768, 2048)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,dim,tokens", GRADS)
def test_embedding_backward(vocab, dim, tokens, dtype):
    g = gen(tokens)
    # by Zipf's law, with the first and last ids and with padding
    ids = (torch.exp(torch.rand(tokens, generator=g, dtype=torch.float64) * np.log(vocab + 1.0)) - 1).long().clamp(0, vocab - 1)
    ids = vocab - 1 - ids if tokens % 2 else ids
    ids[torch.rand(tokens, generator=g) < 0.1] = torch.tensor([-1, vocab])[tokens % 2]
    dy = matrix(tokens, dim, dtype, 3, 0.1)
    want, size, count = sums64(ids, dy, vocab)
    scale = 1.7
    want, size = want * np.float32(scale), size * float(np.float32(scale))
    out = torch.full((vocab, dim), float("nan"), dtype=TD[dtype], device="cuda")
    L.embedding_backward(dy.cuda(), ids.cuda(), out, scale)
    bound = half_step(want, TD[dtype]) + (count + 1) * U * size
    assert within(out, want, torch.where(size > 0, bound, 0.0))
    for _ in range(3):                                  # no order of arrival shows
        again = torch.full_like(out, 3.0)
        L.embedding_backward(dy.cuda(), ids.int().cuda(), again, scale)
        assert torch.equal(again, out)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("offset,gap", LAYOUTS)
def test_embedding_backward_of_whole_numbers_is_exact(offset, gap, accumulate):
    vocab, dim, tokens = 61, 203, 700
    g = gen(7)
    ids = torch.randint(-3, vocab, (tokens,), generator=g)
    ids[100:350] = 17                                   # a run over many pieces
    ids[ids == 40] = 41                                 # a row without tokens
    dy = torch.randint(-2, 3, (tokens, dim), generator=g).half()
    held = torch.randint(-5, 6, (vocab, dim), generator=g).half()
    want = sums64(ids, dy, vocab)[0] * 2 + (held.double() if accumulate else 0)
    assert float(want.abs().max()) < 2048
    out, room = strided(held, offset, gap)
    need = Z.zero_embedding_backward_workspace_bytes(vocab, dim, tokens)
    work = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    src = strided(dy, (offset + 5) % 9, gap)[0]
    L.embedding_backward(src, ids.cuda(), out, 2.0, accumulate, work[:need])
    assert torch.equal(out.double().cpu(), want)
    assert untouched(out, room) and bool((work[need:] == 0xA5).all())


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 31, 32, 33, 512, 1024 * 8, 1024 * 8 + 1, 30000])
def test_embedding_backward_of_one_id(tokens):
    # one run over all pieces, which begins and ends at their edges or inside them; and behind it padding
    dy = torch.ones((tokens, 24), dtype=torch.float16, device="cuda")
    ids = torch.full((tokens,), 3, device="cuda")
    for padded in (0, 1, 5):
        ids[:padded] = -1
        out = torch.full((5, 24), 9.0, dtype=torch.float16, device="cuda")
        L.embedding_backward(dy, ids, out)
        assert bool((out[3] == max(0, tokens - padded)).half().all()) if tokens < 2048 else \
            torch.equal(out[3], torch.full((24,), tokens - padded).half().cuda())
        assert not out[[0, 1, 2, 4]].any()


@pytest.mark.parametrize("vocab", [1, 2, 3, 16, 17, 100, 255, 256, 257, 65535, 65536, 65537, 2 ** 17 - 1])
def test_embedding_backward_sorts_every_id(vocab):
    # each id once, in a shuffled order: rows are the gradients themselves
    perm = torch.randperm(vocab, generator=gen(vocab))
    dy = (torch.arange(vocab * 2).view(vocab, 2) % 2039).half().cuda()
    out = torch.empty_like(dy)
    L.embedding_backward(dy, perm.cuda(), out)
    assert torch.equal(out[perm.cuda()], dy)


def test_embedding_backward_against_differences():
    # the loss sum(out * c) is linear in the table: whole-number steps give the slope itself
    table, ids = torch.randint(-3, 4, (20, 40), generator=gen(1)).half(), torch.randint(0, 20, (64,), generator=gen(2))
    c = torch.randint(-2, 3, (64, 40), generator=gen(3)).half()
    loss = lambda t: float((L.embedding(ids.cuda(), t.cuda(), 2.0).double().cpu() * c.double()).sum())   # noqa: E731
    grad = L.embedding_backward(c.cuda(), ids.cuda(), torch.empty(20, 40, dtype=torch.float16, device="cuda"), 2.0)
    base = loss(table)
    for i, j in ((0, 0), (7, 13), (19, 39)):
        moved = table.clone()
        moved[i, j] += 1
        assert loss(moved) - base == float(grad[i, j])


def test_embedding_past_32_bits():
    vocab, dim = 1_100_003, 4000                        # 4.4e9 elements
    table = torch.zeros((vocab, dim), dtype=torch.bfloat16, device="cuda")
    table[-5:] = matrix(5, dim, "bf16", 1).cuda()
    ids = torch.tensor([vocab - 1, vocab - 5, 0, vocab - 3], device="cuda")
    out = L.embedding(ids, table)
    assert torch.equal(out, table[ids])
    L.embedding_backward(out, ids, table.fill_(7.0))
    assert torch.equal(table[ids], out) and not table[:vocab - 5].any() and not table[vocab - 2].any()
    L.embedding_backward(out, ids, table, accumulate=True)
    assert torch.equal(table[ids].float(), out.float() * 2)


# ------------------------------------------------------------ all of them
def test_empty_calls():
    h = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    w, spec = torch.ones(64, dtype=torch.bfloat16, device="cuda"), Z.dropout_spec(0.1, 1)
    assert L.dropout(h, spec).shape == (0, 64) and L.dropout(h.t().contiguous(), spec).shape == (64, 0)
    n = L.rms_norm(h, w, residual=h, bits=8)
    assert n.h.shape == n.y.shape == (0, 64) and n.q.rows == 0
    dh, dx, dw = L.rms_norm_backward(h, h, w, dweight=w.clone())
    assert dh.shape == (0, 64) and not dw.any()
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    table = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    assert L.embedding(ids, table).shape == (0, 64)
    L.embedding_backward(h, ids, table, accumulate=True)
    assert bool((table == 1).all())
    L.embedding_backward(h, ids, table)
    assert not table.any()


def test_other_stream_and_graph():
    """Everything on a side stream, and captured; the replays' dropout follows the device's step word."""
    rows, cols, vocab = 40, 264, 90
    table, w = matrix(vocab, cols, "bf16", 1).cuda(), matrix(1, cols, "bf16", 2)[0].cuda()
    ids = torch.randint(0, vocab, (rows,), generator=gen(3)).cuda()
    dy = matrix(rows, cols, "bf16", 4).cuda()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(spec, room, room2):
        x = L.embedding(ids, table, 2.0)
        n = L.rms_norm(L.dropout(x, spec), w, residual=x, dropout=spec, bits=8)
        dh, dx, dw = L.rms_norm_backward(dy, n.h, w, dropout=spec, workspace=room)
        dt = L.embedding_backward(L.dropout(dx, spec), ids, torch.empty_like(table), 2.0, workspace=room2)
        return n.h, n.y, n.q.codes[:rows * 288], n.q.scales, dh, dx, dw, dt

    rooms = (torch.empty(Z.zero_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda"),
             torch.empty(Z.zero_embedding_backward_workspace_bytes(vocab, cols, rows), dtype=torch.uint8, device="cuda"))
    want = [run(Z.dropout_spec(0.2, 6, k), *rooms) for k in range(3)]
    assert not torch.equal(want[0][0], want[1][0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(Z.dropout_spec(0.2, 6, 0), *rooms)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    spec = Z.dropout_spec(0.2, 6, 0, step)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]     # they share the workspaces, and run in order
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(run(spec, *rooms))
    for k in (0, 1, 2, 1):
        step.fill_(k)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want[k]))


def test_many_passes_in_a_row():
    # each call's start overlaps the end of the one before it; two streams with workspaces of their own
    rows, cols, vocab = 900, 1000, 5000
    table, w = matrix(vocab, cols, "bf16", 1).cuda(), matrix(1, cols, "bf16", 2)[0].cuda()
    ids = torch.randint(0, vocab, (rows,), generator=gen(3)).cuda()
    spec = Z.dropout_spec(0.1, 6)

    def run(grad):
        x = L.embedding(ids, table)
        n = L.rms_norm(x, w, residual=x, dropout=spec, bits=8)
        dh, dx, dw = L.rms_norm_backward(n.y, n.h, w, dropout=spec)
        return n.q.values(), dh, dx, dw, L.embedding_backward(dx, ids, grad)

    want = run(torch.empty_like(table))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    grads = [torch.empty_like(table) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(60):
        for s, grad in zip(streams, grads):
            with torch.cuda.stream(s):
                got = run(grad)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(grads[0], want[-1])


def test_refusals_with_tensors():
    x, w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    ids, spec = torch.zeros(8, dtype=torch.int64, device="cuda"), Z.dropout_spec(0.1, 1)

    def refused(text, fn, *a, **kw):
        with pytest.raises(Z.ZeroError) as e:
            fn(*a, **kw)
        assert e.value.code == 1 and text in str(e.value), str(e.value)

    refused("fp16 or bf16", L.dropout, x.float(), spec)
    refused("rows", L.dropout, x.t(), spec)
    refused("out must", L.dropout, x, spec, out=x[:4])
    refused("rows", L.dropout, x, spec, out=w.expand(8, 64))
    refused("GPU", L.dropout, x, Z.dropout_spec(0.1, 1, 0, torch.zeros(1, dtype=torch.int64)))
    refused("int64", L.dropout, x, Z.dropout_spec(0.1, 1, 0, torch.zeros(1, device="cuda")))
    refused("p must", L.dropout, x, Z.dropout_spec(1.0, 1))
    refused("weight", L.rms_norm, x, w[:32])
    refused("weight", L.rms_norm, x, w.half())
    refused("residual", L.rms_norm, x, w, residual=x[:4])
    refused("nothing", L.rms_norm, x, w, wide=False)
    refused("bits", L.rms_norm, x, w, bits=16)
    refused("out must", L.rms_norm, x, w, bits=8, out=Mx4Matrix(8, 64))
    refused("out must", L.rms_norm, x, w, bits=8, out=Mx8Matrix(8, 32))
    refused("eps", L.rms_norm, x, w, -1.0)
    refused("dy", L.rms_norm_backward, x[:4], x, w)
    refused("workspace", L.rms_norm_backward, x, x, w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    refused("ids", L.embedding, ids.float(), x)
    refused("ids", L.embedding, ids.view(2, 4).t(), x)
    refused("out must", L.embedding, ids, x, out=x.half())
    refused("dout", L.embedding_backward, x[:4], ids, x.clone())
    refused("workspace", L.embedding_backward, x, ids, x.clone(), workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    refused("columns", L.rms_norm, torch.zeros((1, 16385), dtype=torch.bfloat16, device="cuda"),
            torch.zeros(16385, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()

"""Microscaled 8-bit floats on the GPU against a 64-bit reference.

Codes, scales and the values read back are exact.  A product sums products of
two e4m3 values (8 bits, exact in fp32) and powers of two in fp32 and is
rounded once to 16 bits: half a step a value, 2^-8 (bf16) or 2^-11 (fp16) of
it at most.  Half a step is reached at the low end of a binade only and the
errors are spread evenly, so the 2-norm of the rounding is about
2^-8 / sqrt(3) / 1.4 of the result's; 2^-9 and 2^-11 (where the fp32 sums of some thousand
terms, 2^-24 each of partial sums that may be several times the result, want
room) bound it."""

import numpy as np
import pytest
import torch

from _layer_ref import mx8_decode, mx8_encode
from _matrix_ref import mx4_tile, rel
import zero_partitioned_mixed_gb300 as Z
from zero_partitioned_mixed_gb300.mx4 import Mx4Matrix, mx4_product
from zero_partitioned_mixed_gb300.mx8 import Mx8Matrix, mx8_linear, mx8_linear_backward, mx8_product

pytestmark = pytest.mark.gpu
TD = {"fp16": torch.float16, "bf16": torch.bfloat16}
PRODUCT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -9}


def matrix(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-6, 6, (rows, 1), generator=g).float())
    return x.to(TD[dtype])


def check_encoding(q, x):
    codes, scales = mx8_encode(x.double().numpy())
    assert np.array_equal(q.codes.cpu().numpy()[:codes.size], codes.reshape(-1))
    tiles = mx4_tile(scales)
    assert np.array_equal(q.scales.cpu().numpy()[:tiles.size], tiles)
    return mx8_decode(codes, scales, x.shape[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 128), (7, 257), (129, 130), (64, 300), (257, 96)])
def test_codes_scales_and_values_are_exact(rows, cols, dtype):
    x = matrix(rows, cols, dtype, rows * cols)
    for q, want in ((Mx8Matrix.of(x.cuda()), x), (Mx8Matrix.of(x.cuda(), transpose=True), x.t().contiguous())):
        values = check_encoding(q, want)
        # 4 significant bits of a power-of-two scale: exact, but for those below fp16's smallest
        assert torch.equal(q.values(TD[dtype]).cpu(), torch.from_numpy(values).to(TD[dtype]))


def specials():
    """Blocks of 32: ties, saturation, signed zeros, subnormals of the elements, extremes, infinities, NaN."""
    ties = [256.0] + [s * v for v in (17.0, 19.0, 34.0, 38.0, 68.0, 272.0, 304.0, 432.0) for s in (1, -1)] + [440.0, 447.0, 456.0, 504.0]
    small = [256.0] + [s * k * 2.0 ** -10 for k in range(1, 12) for s in (1, -1)] + [2.0 ** -6, 2.0 ** -11, 3 * 2.0 ** -11]
    rows = [ties, small, [511.0, 480.0, 464.0, 463.0, -511.0], [0.0] * 32, [-0.0] * 32, [1e-30, -1e-31],
            [2.0 ** -133, -(2.0 ** -130)], [2.0 ** -126, 2.0 ** -128], [3.3e38, -1.0, 1e30], [float("inf"), 1.0],
            [1.0, -float("inf")], [2.0, float("nan")], [float("nan")] * 32, [1.0], [-1.5], [2.0 ** -119 * 1.5, 2.0 ** -127]]
    return torch.tensor([r + [0.0] * (32 - len(r)) for r in rows])


def test_special_blocks():
    x = torch.cat((specials(), specials().flip(1)), 1).bfloat16()     # two blocks a row
    for q, want in ((Mx8Matrix.of(x.cuda()), x), (Mx8Matrix.of(x.t().contiguous().cuda(), transpose=True), x)):
        values = check_encoding(q, want)
        got = q.values().double().cpu().numpy()
        expect = torch.from_numpy(values).bfloat16().double().numpy()
        assert np.array_equal(got, expect, equal_nan=True)
        assert np.array_equal(np.signbit(got[~np.isnan(got)]), np.signbit(expect[~np.isnan(expect)]))


def test_every_code_is_read_back():
    q = Mx8Matrix(2, 128)
    codes = np.array([c for c in range(256) if c & 127 != 127] + [0, 128], np.uint8).reshape(2, 128)
    scales = np.array([[127, 120, 130, 127], [127, 127, 119, 140]], np.uint8)
    q.codes.copy_(torch.from_numpy(codes.reshape(-1)))
    q.scales.copy_(torch.from_numpy(mx4_tile(scales)))
    assert np.array_equal(q.values().double().cpu().numpy(), mx8_decode(codes, scales, 128))


@pytest.mark.parametrize("offset,ld", [(0, 104), (1, 97), (8, 99), (5, 104)])
@pytest.mark.parametrize("transpose", [False, True])
def test_strided_sources_and_destinations(offset, ld, transpose):
    rows, cols = 66, 97
    room = torch.full((rows * ld + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = room[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    x = matrix(rows, cols, "bf16", 3)
    view.copy_(x)
    q = Mx8Matrix.of(view, transpose=transpose)
    values = check_encoding(q, x.t().contiguous() if transpose else x)
    if transpose:
        return
    out = torch.full((rows * ld + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    dst = out[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    Z.zero_mx8_dequantize(Z.ZERO_BF16, rows, cols, q.codes, q.scales, dst, ld=ld)
    assert np.array_equal(dst.double().cpu().numpy(), values)
    dst.fill_(5.0)
    assert bool((out == 5.0).all())


def test_code_and_scale_buffers_keep_their_bounds():
    for rows, cols, transpose in ((130, 161, False), (161, 130, True), (1, 1, False), (1, 1, True)):
        r, c = (cols, rows) if transpose else (rows, cols)
        nc, ns = Z.zero_mx8_codes_bytes(r, c), Z.zero_mx8_scales_bytes(r, c)
        codes, scales = (torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda") for n in (nc, ns))
        Z.zero_mx8_quantize(Z.ZERO_BF16, rows, cols, matrix(rows, cols, "bf16", 1).cuda(), codes, scales, transpose=transpose)
        assert bool((codes[nc:] == 0xA5).all()) and bool((scales[ns:] == 0xA5).all())


PRODUCTS = [(1, 1, 1), (1, 300, 64), (1, 129, 1000), (2, 8, 31), (5, 257, 96), (16, 40, 33), (17, 130, 512), (33, 640, 2049),
            (64, 128, 128), (100, 100, 4100), (32, 200, 700), (65, 2000, 300), (127, 129, 257), (128, 256, 256), (130, 515, 1111),
            (300, 70, 640), (513, 511, 300), (700, 1300, 384), (2100, 4000, 520), (257, 193, 64), (3000, 2000, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products_match_64_bits(m, n, k, dtype):
    x, w = torch.randn(m, k, generator=torch.Generator().manual_seed(m)), torch.randn(n, k, generator=torch.Generator().manual_seed(n + k))
    x, w = x.to(TD[dtype]), w.to(TD[dtype])
    qx, qw = Mx8Matrix.of(x.cuda()), Mx8Matrix.of(w.cuda())
    room = torch.full((m * (n + 3) + 8,), 5.0, dtype=TD[dtype], device="cuda")
    outs = [mx8_product(qx, qw, TD[dtype]), room[1:1 + m * (n + 3)].view(m, n + 3)[:, :n]]
    mx8_product(qx, qw, out=outs[1])
    Z.zero_matrix_status()
    want = qx.values(TD[dtype]).double().cpu() @ qw.values(TD[dtype]).double().cpu().t()
    assert rel(outs[0], want) <= PRODUCT[dtype]
    assert torch.equal(outs[0], outs[1])
    outs[1].fill_(5.0)
    assert bool((room == 5.0).all())


def test_exact_products():
    # whole numbers that the format holds under every block's scale: fp32 sums and the 16-bit result are exact
    g = torch.Generator().manual_seed(5)
    vals = torch.tensor([0.0, 1.0, 2.0, 3.0, 5.0, 7.0, -1.0, -6.0])
    for m, n, k in ((1, 200, 320), (20, 70, 130), (40, 72, 256), (260, 130, 1024)):
        x, w = vals[torch.randint(0, 8, (m, k), generator=g)], vals[torch.randint(0, 8, (n, k), generator=g)]
        keep = torch.zeros(k)
        keep[::32] = 1                          # small sums: every result is a whole number below 2048
        got = mx8_linear((x * keep).half().cuda(), Mx8Matrix.of(w.half().cuda()))
        want = (x * keep).double() @ w.double().t()
        assert float(want.abs().max()) < 2048 and torch.equal(got.double().cpu(), want)


def test_each_block_has_its_own_scale():
    # one value a block, each block at another power of two: a scale taken from another block would show
    k = 32 * 12
    x, w = torch.zeros(3, k), torch.zeros(200, k)
    for b in range(12):
        x[:, 32 * b] = 2.0 ** (b % 5) * torch.tensor([1.0, 1.25, -1.5])
        w[:, 32 * b + 0] = (2.0 ** -(b % 5)) * (1 + torch.arange(200) % 8 / 8.0) * (1 if b % 2 else 2)
    for rows in (3, 60, 200):
        xs = x.repeat((rows + 2) // 3, 1)[:rows]
        got = mx8_linear(xs.half().cuda(), Mx8Matrix.of(w.half().cuda()))
        # (1.875, alone in its block, lies above the largest code of its scale and becomes 1.75)
        hold = lambda v: torch.from_numpy(mx8_decode(*mx8_encode(v.double().numpy()), k))   # noqa: E731
        assert torch.equal(got.double().cpu(), hold(xs) @ hold(w).t())


def test_nan_blocks_reach_their_rows_and_columns_only():
    x, w = torch.randn(40, 300).bfloat16(), torch.randn(150, 300).bfloat16()
    clean = mx8_linear(x.cuda(), Mx8Matrix.of(w.cuda()))
    x[3, 299] = float("nan")
    w[149, 0] = float("inf")
    got = mx8_linear(x.cuda(), Mx8Matrix.of(w.cuda()))
    assert torch.isnan(got[3]).all() and torch.isnan(got[:, 149]).all()
    rest = torch.ones(40, 150, dtype=torch.bool, device="cuda")
    rest[3], rest[:, 149] = False, False
    assert torch.equal(got[rest], clean[rest])


def test_scales_over_the_whole_range():
    x, w = torch.ones(4, 64), torch.ones(6, 64)
    x[:, 32:] = 0
    w[:, 32:] = 0
    want = mx8_linear(x.bfloat16().cuda(), Mx8Matrix.of(w.bfloat16().cuda()))
    got = mx8_linear((x * 2.0 ** 100).bfloat16().cuda(), Mx8Matrix.of((w * 2.0 ** -110).bfloat16().cuda()))
    assert torch.equal(want, torch.full_like(want, 32.0)) and torch.equal(got.double(), want.double() * 2.0 ** -10)


def test_empty_products():
    z = torch.zeros(16, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 5), 4.0, dtype=torch.bfloat16, device="cuda")
    Z.zero_mx8_matmul(Z.ZERO_BF16, 3, 5, 0, z, z, z, z, out)
    assert not out.any()
    Z.zero_mx8_matmul(Z.ZERO_BF16, 0, 5, 64, None, None, z, z, None)
    Z.zero_mx8_quantize(Z.ZERO_BF16, 0, 5, None, None, None)
    Z.zero_mx8_dequantize(Z.ZERO_BF16, 4, 0, None, None, None)


def test_linear_layer_and_its_gradients():
    """Against the formulas on the quantised operands, and, on values that the
    format holds exactly, against differences of the loss."""
    t, k, n = 70, 130, 200
    x, w, dy = matrix(t, k, "bf16", 1), matrix(n, k, "bf16", 2), matrix(t, n, "bf16", 3)
    dx, dw = mx8_linear_backward(dy.cuda(), x.cuda(), Mx8Matrix.of(w.cuda(), transpose=True))
    val = lambda a, tr: Mx8Matrix.of(a.cuda(), transpose=tr).values().double().cpu()   # noqa: E731
    assert rel(dx, val(dy, False) @ val(w, True).t()) <= PRODUCT["bf16"]
    assert rel(dw, val(dy, True) @ val(x, True).t()) <= PRODUCT["bf16"]

    g = torch.Generator().manual_seed(4)
    vals = torch.tensor([0.0, 1.0, -1.0, 2.0])
    pick = lambda *s: vals[torch.randint(0, 4, s, generator=g)]   # noqa: E731
    x, w, dy = pick(t, k), pick(n, k), pick(t, n)
    dx, dw = mx8_linear_backward(dy.half().cuda(), x.half().cuda(), Mx8Matrix.of(w.half().cuda(), transpose=True))

    def loss(x, w):
        y = mx8_linear(x.half().cuda(), Mx8Matrix.of(w.half().cuda()))
        return float((y.double().cpu() * dy.double()).sum())

    base = loss(x, w)
    for i, j in ((0, 0), (69, 129), (35, 64)):
        moved = x.clone()
        moved[i, j] += 1      # stays a value of the format, and the loss is linear in it
        assert loss(moved, w) - base == float(dx[i, j])
    for i, j in ((0, 0), (199, 129), (100, 31)):
        moved = w.clone()
        moved[i, j] += 1
        assert loss(x, moved) - base == float(dw[i, j])


def test_other_stream_graph_and_repeats():
    x, w = matrix(50, 500, "bf16", 1).cuda(), Mx8Matrix.of(matrix(300, 500, "bf16", 2).cuda())
    want = mx8_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mx8_linear(x, w)
    s.synchronize()
    assert torch.equal(got, want)
    scratch, out = Mx8Matrix(50, 500), torch.zeros_like(want)
    src, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx8_linear(src, w, out, scratch)
    src.copy_(x)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_past_32_bits():
    rows, cols, tail = 66016, 66003, 160        # 4.36e9 values, rows at odd offsets; the tail is whole blocks
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-tail:] = matrix(tail, cols, "bf16", 1).cuda()
    q, small = Mx8Matrix.of(x), Mx8Matrix.of(x[-tail:])
    assert torch.equal(q.codes.view(rows, -1)[-tail:], small.codes.view(tail, -1))
    y = q.values()
    assert torch.equal(y[-tail:], small.values()) and not y[:-tail].any()
    y = Mx8Matrix.of(x, transpose=True).values()
    assert torch.equal(y[:, -tail:], Mx8Matrix.of(x[-tail:], transpose=True).values()) and not y[:, :-tail].any()
    del y
    w = Mx8Matrix.of(matrix(70, cols, "bf16", 2).cuda())
    out = mx8_product(q, w)                     # the last rows' codes lie beyond 2^32 bytes
    # (two results, each within 2^-9 of the exact one)
    assert rel(out[-tail:], mx8_product(small, w).double().cpu()) <= 2.0 ** -8 and not out[:-tail].any()


def test_many_passes_in_a_row():
    # quantising and product alternate without a wait for the host, each overlapping the other's start
    x, w = matrix(1500, 1024, "bf16", 1).cuda(), Mx8Matrix.of(matrix(3000, 1024, "bf16", 2).cuda())
    few = x[:7]
    want, want_few = mx8_linear(x, w), mx8_linear(few, w)
    scratch, scratch_few = Mx8Matrix(1500, 1024), Mx8Matrix(7, 1024)
    outs, outs_few = [torch.empty_like(want) for _ in range(4)], [torch.empty_like(want_few) for _ in range(4)]
    for i in range(400):
        mx8_linear(x, w, outs[i % 4], scratch)
        mx8_linear(few, w, outs_few[i % 4], scratch_few)
    Z.zero_matrix_status()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(o, want_few) for o in outs_few)


def test_matrices_of_an_optimizer_s_replicas():
    from zero_partitioned_mixed_gb300.muon import MuonBuffers
    buf = MuonBuffers([(40, 70), (33, 128)], 2, "bf16")
    x = matrix(33, 128, "bf16", 1)
    buf.matrix(1, buf.params[1]).copy_(x)
    for transpose in (False, True):
        q = buf.quantize(1, transpose, rank=1, bits=8)
        assert isinstance(q, Mx8Matrix)
        check_encoding(q, x.t().contiguous() if transpose else x)
        assert torch.equal(buf.quantize(1, transpose, 1).codes, Mx4Matrix.of(x.cuda(), transpose).codes)
    with pytest.raises(Z.ZeroError) as e:
        buf.quantize(0, bits=16)
    assert e.value.code == 1 and "bits" in str(e.value)


def test_refusals():
    z = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    h = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")

    def refused(text, fn, *a, **kw):
        with pytest.raises(Z.ZeroError) as e:
            fn(*a, **kw)
        assert e.value.code == 1 and text in str(e.value), str(e.value)

    refused("dtype", Z.zero_mx8_quantize, 3, 4, 32, h, z, z)
    refused("codes", Z.zero_mx8_quantize, 1, 4, 32, h, z[1:], z)
    refused("scales", Z.zero_mx8_quantize, 1, 4, 32, h, z, None)
    refused("ld", Z.zero_mx8_quantize, 1, 4, 32, h, z, z, ld=31)
    refused("out16", Z.zero_mx8_dequantize, 1, 4, 32, z, z, None)
    refused("codes", Z.zero_mx8_matmul, 1, 4, 4, 32, None, z, z, z, h)
    refused("ld", Z.zero_mx8_matmul, 1, 4, 4, 32, z, z, z, z, h, ld=3)
    refused("columns", mx8_product, Mx8Matrix(2, 32), Mx8Matrix(2, 64))
    # codes of one width are not those of the other
    refused("Mx8Matrix", mx8_product, Mx8Matrix(2, 32), Mx4Matrix(2, 32))
    refused("Mx4Matrix", mx4_product, Mx8Matrix(2, 32), Mx4Matrix(2, 32))
    refused("Mx8Matrix", mx8_linear, h.view(64, 64), Mx4Matrix(2, 64))
    refused("fp16 or bf16", Mx8Matrix.of, torch.zeros(4, 4, device="cuda"))
    refused("contiguous rows", Mx8Matrix.of, h.view(64, 64).t())
    torch.cuda.synchronize()


@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (20, 129, 300), (32, 200, 5000), (100, 600, 1300), (2100, 4000, 520)])
@pytest.mark.parametrize("stage", [0, 1])
def test_a_wait_that_runs_out_ends_the_call_and_is_reported(m, n, k, stage):
    """All forms of the product: block 0 stops copying its operands on purpose."""
    qx, qw = Mx8Matrix.of(matrix(m, k, "bf16", 1).cuda()), Mx8Matrix.of(matrix(n, k, "bf16", 2).cuda())
    want = mx8_product(qx, qw)
    room = torch.full((m * n + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[256:256 + m * n].view(m, n)
    Z._binding.zero_debug_hold_matrix(stage)
    mx8_product(qx, qw, out=out)
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_matrix_status()
    assert e.value.code == 4 and "zero_mx8_matmul" in str(e.value)
    for _ in range(2):
        mx8_product(qx, qw, out=out)
    Z.zero_matrix_status()
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((room == 7.0).all())

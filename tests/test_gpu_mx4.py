"""Microscaled 4-bit floats on the GPU against a 64-bit reference.

Codes, scales and the values read back are exact.  A product sums exact
fp32 products of at most 36 x 2^e in fp32 and is rounded once to 16 bits:
2^-9 (bf16) or 2^-12 (fp16) a value at most, 2-norm about 0.6 of that, so
2^-9 and 2^-11 (room for the fp32 sums of some thousand terms) bound it."""

import numpy as np
import pytest
import torch

from _matrix_ref import mx4_decode, mx4_encode, mx4_pack, mx4_tile, rel
import zero_partitioned_mixed_gb300 as Z
from zero_partitioned_mixed_gb300.mx4 import Mx4Matrix, mx4_linear, mx4_linear_backward, mx4_product

pytestmark = pytest.mark.gpu
TD = {"fp16": torch.float16, "bf16": torch.bfloat16}
PRODUCT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -9}


def matrix(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-6, 6, (rows, 1), generator=g).float())
    return x.to(TD[dtype])


def check_encoding(q, x):
    codes, scales = mx4_encode(x.double().numpy())
    packed = mx4_pack(codes)
    assert np.array_equal(q.codes.cpu().numpy()[:packed.size], packed.reshape(-1))
    tiles = mx4_tile(scales)
    assert np.array_equal(q.scales.cpu().numpy()[:tiles.size], tiles)
    return mx4_decode(codes, scales, x.shape[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 128), (7, 257), (129, 130), (64, 1000), (257, 96)])
def test_codes_scales_and_values_are_exact(rows, cols, dtype):
    x = matrix(rows, cols, dtype, rows * cols)
    for q, want in ((Mx4Matrix.of(x.cuda()), x), (Mx4Matrix.of(x.cuda(), transpose=True), x.t().contiguous())):
        values = check_encoding(q, want)
        # (2 significant bits of a power-of-two scale: exact in both types unless it leaves fp16's range)
        assert np.array_equal(q.values(TD[dtype]).double().cpu().numpy(), values)


def specials():
    """Blocks of 32: ties, saturation, signed zeros, subnormals, extremes, infinities, NaN."""
    grid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    ties = [4.0] + [s * v for v in grid for s in (1, -1)] + [0.2490234375, 0.251953125, 6.99, -7.5]
    rows = [ties, [7.0, 6.5, -7.9, 1.0], [0.0] * 32, [-0.0] * 32, [1e-30, -1e-31], [2.0 ** -133, -(2.0 ** -130)],
            [2.0 ** -126, 2.0 ** -128], [3.3e38, -1.0, 1e30], [float("inf"), 1.0], [1.0, -float("inf")],
            [2.0, float("nan")], [float("nan")] * 32, [1.0], [-1.5], [2.0 ** -125 * 1.5]]
    return torch.tensor([r + [0.0] * (32 - len(r)) for r in rows])


def test_special_blocks():
    x = torch.cat((specials(), specials().flip(1)), 1).bfloat16()     # two blocks a row
    for q, want in ((Mx4Matrix.of(x.cuda()), x), (Mx4Matrix.of(x.t().contiguous().cuda(), transpose=True), x)):
        values = check_encoding(q, want)
        got = q.values().double().cpu().numpy()
        expect = torch.from_numpy(values).bfloat16().double().numpy()
        assert np.array_equal(got, expect, equal_nan=True)
        assert np.array_equal(np.signbit(got[~np.isnan(got)]), np.signbit(expect[~np.isnan(expect)]))


def test_fp16_values_at_the_formats_limits():
    x = torch.tensor([[65504.0, -65504.0, 6.0e-8, 1.0], [6.0e-8, -6.0e-8, 1.2e-7, 0.0]], dtype=torch.float16)
    q = Mx4Matrix.of(x.cuda())
    values = check_encoding(q, x)
    assert np.array_equal(q.values(torch.float16).double().cpu().numpy(), torch.from_numpy(values).half().double().numpy())


@pytest.mark.parametrize("offset,ld", [(0, 104), (1, 97), (8, 99), (5, 104)])
@pytest.mark.parametrize("transpose", [False, True])
def test_strided_sources_and_destinations(offset, ld, transpose):
    rows, cols = 66, 97
    room = torch.full((rows * ld + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = room[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    x = matrix(rows, cols, "bf16", 3)
    view.copy_(x)
    q = Mx4Matrix.of(view, transpose=transpose)
    values = check_encoding(q, x.t().contiguous() if transpose else x)
    if transpose:
        return
    out = torch.full((rows * ld + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    dst = out[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    Z.zero_mx4_dequantize(Z.ZERO_BF16, rows, cols, q.codes, q.scales, dst, ld=ld)
    assert np.array_equal(dst.double().cpu().numpy(), values)
    dst.fill_(5.0)
    assert bool((out == 5.0).all())


def test_code_and_scale_buffers_keep_their_bounds():
    for rows, cols, transpose in ((130, 161, False), (161, 130, True), (1, 1, False), (1, 1, True)):
        r, c = (cols, rows) if transpose else (rows, cols)
        nc, ns = Z.zero_mx4_codes_bytes(r, c), Z.zero_mx4_scales_bytes(r, c)
        codes, scales = (torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda") for n in (nc, ns))
        Z.zero_mx4_quantize(Z.ZERO_BF16, rows, cols, matrix(rows, cols, "bf16", 1).cuda(), codes, scales, transpose=transpose)
        assert bool((codes[nc:] == 0xA5).all()) and bool((scales[ns:] == 0xA5).all())


PRODUCTS = [(1, 1, 1), (1, 300, 64), (1, 129, 1000), (2, 8, 31), (5, 257, 96), (16, 40, 33), (17, 130, 512), (33, 640, 2049),
            (64, 128, 128), (100, 100, 4100), (32, 200, 700), (65, 2000, 300), (127, 129, 257), (128, 256, 256), (130, 515, 1111), (300, 70, 640),
            (513, 511, 300), (700, 1300, 384), (2100, 4000, 520), (257, 193, 64), (3000, 2000, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products_match_64_bits(m, n, k, dtype):
    x, w = torch.randn(m, k, generator=torch.Generator().manual_seed(m)), torch.randn(n, k, generator=torch.Generator().manual_seed(n + k))
    x, w = x.to(TD[dtype]), w.to(TD[dtype])
    qx, qw = Mx4Matrix.of(x.cuda()), Mx4Matrix.of(w.cuda())
    room = torch.full((m * (n + 3) + 8,), 5.0, dtype=TD[dtype], device="cuda")
    outs = [mx4_product(qx, qw, TD[dtype]), room[1:1 + m * (n + 3)].view(m, n + 3)[:, :n]]
    mx4_product(qx, qw, out=outs[1])
    Z.zero_matrix_status()
    want = qx.values(TD[dtype]).double().cpu() @ qw.values(TD[dtype]).double().cpu().t()
    assert rel(outs[0], want) <= PRODUCT[dtype]
    assert torch.equal(outs[0], outs[1])
    outs[1].fill_(5.0)
    assert bool((room == 5.0).all())


def test_exact_products():
    # whole numbers that the format holds: fp32 sums and the 16-bit result are exact
    g = torch.Generator().manual_seed(5)
    vals = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0, -1.0, -2.0])
    for m, n, k in ((1, 200, 320), (40, 72, 256), (260, 130, 1024)):
        x, w = vals[torch.randint(0, 8, (m, k), generator=g)], vals[torch.randint(0, 8, (n, k), generator=g)]
        x[:, ::32], w[:, ::32] = 4.0, 4.0       # every block's scale is 1
        keep = torch.zeros(k)
        keep[::16] = 1                          # small sums: every result is a whole number below 2048
        got = mx4_linear((x * keep).half().cuda(), Mx4Matrix.of(w.half().cuda()))
        want = (x * keep).double() @ w.double().t()
        assert float(want.abs().max()) < 2048 and torch.equal(got.double().cpu(), want)


def test_nan_blocks_reach_their_rows_and_columns_only():
    x, w = torch.randn(40, 300).bfloat16(), torch.randn(150, 300).bfloat16()
    clean = mx4_linear(x.cuda(), Mx4Matrix.of(w.cuda()))
    x[3, 299] = float("nan")
    w[149, 0] = float("inf")
    got = mx4_linear(x.cuda(), Mx4Matrix.of(w.cuda()))
    assert torch.isnan(got[3]).all() and torch.isnan(got[:, 149]).all()
    rest = torch.ones(40, 150, dtype=torch.bool, device="cuda")
    rest[3], rest[:, 149] = False, False
    assert torch.equal(got[rest], clean[rest])


def test_scales_over_the_whole_range():
    # products of very large with very small blocks: the scales multiply as powers of two
    x, w = torch.ones(4, 64), torch.ones(6, 64)
    x[:, 32:] = 0
    w[:, 32:] = 0
    want = mx4_linear(x.bfloat16().cuda(), Mx4Matrix.of(w.bfloat16().cuda()))
    got = mx4_linear((x * 2.0 ** 100).bfloat16().cuda(), Mx4Matrix.of((w * 2.0 ** -110).bfloat16().cuda()))
    assert torch.equal(want, torch.full_like(want, 32.0)) and torch.equal(got.double(), want.double() * 2.0 ** -10)


def test_empty_products():
    z = torch.zeros(16, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 5), 4.0, dtype=torch.bfloat16, device="cuda")
    Z.zero_mx4_matmul(Z.ZERO_BF16, 3, 5, 0, z, z, z, z, out)
    assert not out.any()
    Z.zero_mx4_matmul(Z.ZERO_BF16, 0, 5, 64, None, None, z, z, None)
    Z.zero_mx4_quantize(Z.ZERO_BF16, 0, 5, None, None, None)
    Z.zero_mx4_dequantize(Z.ZERO_BF16, 4, 0, None, None, None)


def test_linear_layer_and_its_gradients():
    """Against the formulas on the quantised operands, and, on values that the
    format holds exactly, against differences of the loss."""
    t, k, n = 70, 130, 200
    x, w, dy = matrix(t, k, "bf16", 1), matrix(n, k, "bf16", 2), matrix(t, n, "bf16", 3)
    dx, dw = mx4_linear_backward(dy.cuda(), x.cuda(), Mx4Matrix.of(w.cuda(), transpose=True))
    val = lambda a, tr: Mx4Matrix.of(a.cuda(), transpose=tr).values().double().cpu()   # noqa: E731
    assert rel(dx, val(dy, False) @ val(w, True).t()) <= PRODUCT["bf16"]
    assert rel(dw, val(dy, True) @ val(x, True).t()) <= PRODUCT["bf16"]

    g = torch.Generator().manual_seed(4)
    vals = torch.tensor([0.0, 1.0, -1.0, 2.0])
    pick = lambda *s: vals[torch.randint(0, 4, s, generator=g)]   # noqa: E731
    x, w, dy = pick(t, k), pick(n, k), pick(t, n)
    dx, dw = mx4_linear_backward(dy.half().cuda(), x.half().cuda(), Mx4Matrix.of(w.half().cuda(), transpose=True))

    def loss(x, w):
        y = mx4_linear(x.half().cuda(), Mx4Matrix.of(w.half().cuda()))
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
    x, w = matrix(50, 500, "bf16", 1).cuda(), Mx4Matrix.of(matrix(300, 500, "bf16", 2).cuda())
    want = mx4_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mx4_linear(x, w)
    s.synchronize()
    assert torch.equal(got, want)
    scratch, out = Mx4Matrix(50, 500), torch.zeros_like(want)
    src, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx4_linear(src, w, out, scratch)
    src.copy_(x)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_past_32_bits():
    rows, cols, tail = 66016, 66003, 160        # 4.36e9 values, rows at odd offsets; the tail is whole blocks
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-tail:] = matrix(tail, cols, "bf16", 1).cuda()
    q, small = Mx4Matrix.of(x), Mx4Matrix.of(x[-tail:])
    assert torch.equal(q.codes.view(rows, -1)[-tail:], small.codes.view(tail, -1))
    y = q.values()
    assert torch.equal(y[-tail:], small.values()) and not y[:-tail].any()
    y = Mx4Matrix.of(x, transpose=True).values()
    assert torch.equal(y[:, -tail:], Mx4Matrix.of(x[-tail:], transpose=True).values()) and not y[:, :-tail].any()
    del y
    w = Mx4Matrix.of(matrix(70, cols, "bf16", 2).cuda())
    out = mx4_product(q, w)                     # the last rows' codes lie beyond 2^31 bytes
    # (two results, each within 2^-9 of the exact one)
    assert rel(out[-tail:], mx4_product(small, w).double().cpu()) <= 2.0 ** -8 and not out[:-tail].any()


def test_many_passes_in_a_row():
    # quantising and product alternate without a wait for the host, each overlapping the other's start
    x, w = matrix(1500, 1024, "bf16", 1).cuda(), Mx4Matrix.of(matrix(3000, 1024, "bf16", 2).cuda())
    few = x[:7]
    want, want_few = mx4_linear(x, w), mx4_linear(few, w)
    scratch, scratch_few = Mx4Matrix(1500, 1024), Mx4Matrix(7, 1024)
    outs, outs_few = [torch.empty_like(want) for _ in range(4)], [torch.empty_like(want_few) for _ in range(4)]
    for i in range(400):
        mx4_linear(x, w, outs[i % 4], scratch)
        mx4_linear(few, w, outs_few[i % 4], scratch_few)
    Z.zero_matrix_status()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(o, want_few) for o in outs_few)


def test_refusals():
    z = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    h = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")

    def refused(text, fn, *a, **kw):
        with pytest.raises(Z.ZeroError) as e:
            fn(*a, **kw)
        assert e.value.code == 1 and text in str(e.value), str(e.value)

    refused("dtype", Z.zero_mx4_quantize, 3, 4, 32, h, z, z)
    refused("codes", Z.zero_mx4_quantize, 1, 4, 32, h, z[1:], z)
    refused("scales", Z.zero_mx4_quantize, 1, 4, 32, h, z, None)
    refused("src16", Z.zero_mx4_quantize, 1, 4, 32, None, z, z)
    refused("ld", Z.zero_mx4_quantize, 1, 4, 32, h, z, z, ld=31)
    refused("2^30", Z.zero_mx4_quantize, 1, (1 << 30) + 1, 32, h, z, z)
    refused("out16", Z.zero_mx4_dequantize, 1, 4, 32, z, z, None)
    refused("ld", Z.zero_mx4_dequantize, 1, 4, 32, z, z, h, ld=5)
    refused("codes", Z.zero_mx4_matmul, 1, 4, 4, 32, None, z, z, z, h)
    refused("scales", Z.zero_mx4_matmul, 1, 4, 4, 32, z, z, z, z[8:], h)
    refused("out16", Z.zero_mx4_matmul, 1, 4, 4, 32, z, z, z, z, None)
    refused("ld", Z.zero_mx4_matmul, 1, 4, 4, 32, z, z, z, z, h, ld=3)
    with pytest.raises(Z.ZeroError):
        mx4_product(Mx4Matrix(2, 32), Mx4Matrix(2, 64))
    with pytest.raises(Z.ZeroError):
        Mx4Matrix(2, 32).fill(h.view(64, 64))
    with pytest.raises(Z.ZeroError):
        Mx4Matrix.of(torch.zeros(4, 4, device="cuda"))
    with pytest.raises(Z.ZeroError):
        Mx4Matrix.of(h.view(64, 64).t())
    torch.cuda.synchronize()


def test_rows_that_share_memory_are_refused():
    # the gradient of y.sum(0) among them: one row for all, so its storage is shorter than its shape
    dy, x, w = torch.zeros(64).bfloat16().cuda().expand(100, 64), matrix(100, 96, "bf16", 1).cuda(), matrix(64, 96, "bf16", 2).cuda()
    q, w_t = Mx4Matrix.of(x), Mx4Matrix.of(w, transpose=True)
    one = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: Mx4Matrix.of(dy), lambda: Mx4Matrix.of(dy, transpose=True), lambda: mx4_linear_backward(dy, x, w_t),
                 lambda: mx4_product(q, Mx4Matrix.of(w), out=one.expand(100, 64))):
        with pytest.raises(Z.ZeroError) as e:
            call()
        assert e.value.code == 1 and "contiguous rows" in str(e.value)
    dx, dw = mx4_linear_backward(dy.contiguous(), x, w_t)
    assert dx.shape == x.shape and dw.shape == w.shape
    torch.cuda.synchronize()


@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (20, 129, 300), (32, 200, 5000), (100, 600, 1300), (2100, 4000, 520)])
@pytest.mark.parametrize("stage", [0, 1])
def test_a_wait_that_runs_out_ends_the_call_and_is_reported(m, n, k, stage):
    """All forms of the product: block 0 stops copying its operands on purpose."""
    qx, qw = Mx4Matrix.of(matrix(m, k, "bf16", 1).cuda()), Mx4Matrix.of(matrix(n, k, "bf16", 2).cuda())
    want = mx4_product(qx, qw)
    room = torch.full((m * n + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[256:256 + m * n].view(m, n)
    Z._binding.zero_debug_hold_matrix(stage)
    mx4_product(qx, qw, out=out)
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_matrix_status()
    assert e.value.code == 4 and "zero_mx4_matmul" in str(e.value)
    for _ in range(2):
        mx4_product(qx, qw, out=out)
    Z.zero_matrix_status()
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((room == 7.0).all())

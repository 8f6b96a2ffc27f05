"""Host-only checks of the residual stream's operators and of microscaled 8-bit
floats (no GPU): sizes, refusals before any CUDA call, and the references
themselves against published values and small cases by hand."""

import numpy as np
import pytest
import torch

from _layer_ref import DECODE, E4M3, dropped, e4m3_code, kept, mx8_encode, norm64, norm_grad64, philox


@pytest.fixture(scope="module")
def Z():
    from zero_partitioned_mixed_gb300.build import build_library
    build_library()
    import zero_partitioned_mixed_gb300 as Z
    return Z


def test_sizes(Z):
    assert Z.zero_mx8_codes_bytes(3, 33) == 3 * 64 and Z.zero_mx8_scales_bytes(129, 129) == 4 * 512
    assert Z.zero_mx8_codes_bytes(10, 0) == 0 and Z.zero_mx8_codes_bytes((1 << 30) + 1, 1) == 0
    assert Z.zero_rms_norm_backward_workspace_bytes(0, 5) == 0 == Z.zero_rms_norm_backward_workspace_bytes(5, 16385)
    assert Z.zero_rms_norm_backward_workspace_bytes(1, 5) == 8 * 4
    assert Z.zero_embedding_backward_workspace_bytes(5, 3, 0) == 0 == Z.zero_embedding_backward_workspace_bytes(0, 3, 5)
    # four arrays of whole numbers, and two partial rows for each piece of tokens
    assert Z.zero_embedding_backward_workspace_bytes(5, 3, 1) >= 16 + 2 * 8 * 4
    import ctypes
    assert ctypes.sizeof(Z._binding.Dropout) == 32


def test_philox_reference_against_published_vectors():
    # the known answers of the paper's own distribution, philox4x32 with 10 rounds
    assert philox(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFFFFFFFFFF
    assert philox(ones, ones, ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert philox(0xA4093822 | 0x299F31D0 << 32, 0x13198A2E | 0x03707344 << 32, 0x243F6A88 | 0x85A308D3 << 32) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_reference():
    keep, factor = kept(3, 11, 0.25, 1, 2)
    words = philox(1, 2, 2 * 2 + 1)                       # row 2, columns 8 to 10
    assert [bool(b) for b in keep[2, 8:]] == [words[0] & 0xFFFF >= 16384, words[0] >> 16 >= 16384, words[1] & 0xFFFF >= 16384]
    assert factor == float(np.float32(65536 / 49152))
    assert kept(1, 8, 1 - 1e-9, 1, 2)[1] == 65536.0 and kept(1, 8, 1e-9, 1, 2)[0].all()
    assert not dropped(torch.full((3, 11), float("nan")), (keep, factor))[~keep].any()


def test_e4m3_reference():
    assert E4M3[126] == 448 and E4M3[8] == 2.0 ** -6 and E4M3[1] == 2.0 ** -9 and E4M3[56] == 1.0
    assert (np.diff(E4M3) > 0).all()
    assert [int(e4m3_code(v)) for v in (17.0, 19.0, 1e9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0)] == [88, 90, 126, 0, 2, 0]
    codes, scales = mx8_encode(np.array([[7.0, -5.0, 0.0, 2.0 ** -20, float(2 ** -3)]]))
    assert scales.tolist() == [[127 + 2 - 8]] and DECODE[8](codes, scales, 5).tolist() == [[7.0, -5.0, 0.0, 0.0, 0.125]]
    assert mx8_encode(np.array([[1.0, np.inf]]))[1].tolist() == [[255]]


def test_norm_references_agree_with_autograd():
    h, w = torch.randn(3, 17, dtype=torch.float64, requires_grad=True), torch.randn(17, dtype=torch.float64, requires_grad=True)
    dy, d = torch.randn(3, 17, dtype=torch.float64), torch.randn(3, 17, dtype=torch.float64)
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-3) * w
    ((y * dy).sum() + (h * d).sum()).backward()
    assert torch.allclose(norm64(h, w, 1e-3)[0], y)
    dh, dw, _, _ = norm_grad64(dy, h.detach(), w.detach(), 1e-3, d)
    assert torch.allclose(dh, h.grad) and torch.allclose(dw, w.grad)


def refused(Z, text, fn, *a, **kw):
    with pytest.raises(Z.ZeroError) as e:
        fn(*a, **kw)
    assert e.value.code == 1 and text in str(e.value), str(e.value)


def test_refusals_come_before_any_cuda_call(Z):
    """Addresses that no call may touch: every refusal has to come first."""
    d = Z.dropout_spec(0.1, 1)
    refused(Z, "dtype", Z.zero_dropout, 2, 4, 8, 16, 16, d, stream=0)
    refused(Z, "src16", Z.zero_dropout, 1, 4, 8, None, 16, d, stream=0)
    refused(Z, "out16 is not", Z.zero_dropout, 1, 4, 8, 16, 17, d, stream=0)
    refused(Z, "ld of src16", Z.zero_dropout, 1, 4, 8, 16, 16, d, ld_src=7, stream=0)
    refused(Z, "step", Z.zero_dropout, 1, 4, 8, 16, 16, Z.dropout_spec(0.1, 1, 0, 12), stream=0)
    refused(Z, "2^30", Z.zero_dropout, 1, (1 << 30) + 1, 8, 16, 16, d, stream=0)
    refused(Z, "together", Z.zero_dropout, 1, 1 << 30, 1 << 39, 16, 16, d, stream=0)
    for p in (1.0, -0.1, float("nan"), float("inf")):
        refused(Z, "p must", Z.zero_dropout, 1, 4, 8, 16, 16, Z.dropout_spec(p, 1), stream=0)
    norm = lambda *a, **kw: Z.zero_rms_norm(*a, stream=0, **kw)   # noqa: E731
    refused(Z, "dtype", norm, 9, 4, 8, 16, 16, 1e-5, out16=16)
    refused(Z, "columns", norm, 1, 4, 16385, 16, 16, 1e-5, out16=16)
    refused(Z, "eps", norm, 1, 4, 8, 16, 16, float("nan"), out16=16)
    refused(Z, "bits", norm, 1, 4, 8, 16, 16, 1e-5, bits=5, codes=16, scales=16)
    refused(Z, "codes", norm, 1, 4, 8, 16, 16, 1e-5, bits=8, codes=8, scales=16)
    refused(Z, "scales", norm, 1, 4, 8, 16, 16, 1e-5, bits=4, codes=16)
    refused(Z, "nothing", norm, 1, 4, 8, 16, 16, 1e-5)
    refused(Z, "weight16", norm, 1, 4, 8, 16, None, 1e-5, out16=16)
    refused(Z, "ld of residual16", norm, 1, 4, 8, 16, 16, 1e-5, residual16=16, ld_residual=3, out16=16)
    back = lambda *a, **kw: Z.zero_rms_norm_backward(*a, stream=0, **kw)   # noqa: E731
    refused(Z, "dy16", back, 1, 4, 8, None, 16, 16, 1e-5, 16)
    refused(Z, "dh16 is NULL", back, 1, 4, 8, 16, 16, 16, 1e-5, None)
    refused(Z, "two matrices", back, 1, 4, 8, 16, 16, 16, 1e-5, 16, dx16=16)
    refused(Z, "workspace", back, 1, 4, 8, 16, 16, 16, 1e-5, 16, dweight16=16)
    refused(Z, "dweight16", back, 1, 4, 8, 16, 16, 16, 1e-5, 16, dweight16=17)
    emb = lambda *a, **kw: Z.zero_embedding(*a, stream=0, **kw)   # noqa: E731
    refused(Z, "vocab", emb, 1, 0, 8, 16, 4, 16, 16)
    refused(Z, "dim", emb, 1, 5, (1 << 20) + 1, 16, 4, 16, 16)
    refused(Z, "tokens", emb, 1, 5, 8, 16, (1 << 31) + 1, 16, 16)
    refused(Z, "ids", emb, 1, 5, 8, 16, 4, 12, 16)
    refused(Z, "id_bytes", emb, 1, 5, 8, 16, 4, torch.zeros(4), 16)
    refused(Z, "scale", emb, 1, 5, 8, 16, 4, 16, 16, scale=float("inf"))
    refused(Z, "table16", emb, 1, 5, 8, 17, 4, 16, 16)
    refused(Z, "ld of out16", emb, 1, 5, 8, 16, 4, 16, 16, ld_out=7)
    grad = lambda *a, **kw: Z.zero_embedding_backward(*a, stream=0, **kw)   # noqa: E731
    refused(Z, "dtable16", grad, 1, 5, 8, 16, 4, 16, None, None)
    refused(Z, "dout16", grad, 1, 5, 8, None, 4, 16, 16, None)
    refused(Z, "workspace is NULL", grad, 1, 5, 8, 16, 4, 16, 16, None)
    refused(Z, "smaller", grad, 1, 5, 8, 16, 4, 16, 16, _Room(256, 64))
    refused(Z, "codes", Z.zero_mx8_quantize, 1, 4, 32, 16, None, 16, stream=0)
    refused(Z, "dtype", Z.zero_mx8_matmul, 9, 4, 4, 32, 16, 16, 16, 16, 16, stream=0)


class _Room:
    """Stands for a tensor at an address: the calls look at no more of a workspace."""

    def __init__(self, at, size):
        self.at, self.size = at, size

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.size

    def element_size(self):
        return 1


def test_tensors_in_host_memory_and_graphs_are_refused(Z):
    from zero_partitioned_mixed_gb300 import layers as L
    from zero_partitioned_mixed_gb300.mx8 import Mx8Matrix, mx8_linear
    x, w, ids = torch.zeros(4, 32).bfloat16(), torch.zeros(32).bfloat16(), torch.zeros(4, dtype=torch.int64)
    m = Mx8Matrix(4, 32, device="cpu")
    for call in (lambda: L.dropout(x, Z.dropout_spec(0.1, 1)), lambda: L.rms_norm(x, w), lambda: L.rms_norm_backward(x, x, w),
                 lambda: L.embedding(ids, x), lambda: L.embedding_backward(x, ids, x), lambda: Mx8Matrix.of(x), m.values,
                 lambda: mx8_linear(x, m), lambda: mx8_linear(m, m)):
        refused(Z, "GPU", call)
    g, v = x.clone().requires_grad_(), w.clone().requires_grad_()
    for call in (lambda: L.dropout(g, Z.dropout_spec(0.1, 1)), lambda: L.rms_norm(g, w), lambda: L.rms_norm(x, v),
                 lambda: L.rms_norm(x, w, residual=g), lambda: L.rms_norm_backward(g, x, w), lambda: L.embedding(ids, g),
                 lambda: L.embedding_backward(g, ids, x), lambda: mx8_linear(g, m), lambda: L.embedding(ids, x, out=g),
                 lambda: L.dropout(x, Z.dropout_spec(0.1, 1), out=g)):
        refused(Z, "autograd", call)
        with torch.no_grad():
            refused(Z, "GPU", call)


def test_shapes_are_refused(Z):
    from zero_partitioned_mixed_gb300 import layers as L
    x = torch.zeros(4, 6, 32).bfloat16()
    refused(Z, "rows", L._matrix, x.transpose(0, 1))
    refused(Z, "one dimension", L._matrix, x[0, 0, 0])
    refused(Z, "contiguous", L._room, torch.zeros(1, dtype=torch.uint8).expand(4096), 4096, "cpu")
    assert L._matrix(x).shape == (24, 32) and L._matrix(x[0, 0]).shape == (1, 32) and L._matrix(x[:, :0]).shape == (0, 32)
    assert L._matrix(x[..., :0]).shape == (24, 0)
    refused(Z, "weight", L._vector, "weight", torch.zeros(8).bfloat16()[::2], 4, torch.bfloat16)


def test_forward_mode_tangents_are_refused(Z):
    """No call gives a result without the tangent that its input had; detached tensors pass on to the next check."""
    from torch.autograd import forward_ad
    from zero_partitioned_mixed_gb300 import layers as L
    from zero_partitioned_mixed_gb300.mx4 import Mx4Matrix, mx4_linear, mx4_linear_backward, mx4_product
    from zero_partitioned_mixed_gb300.mx8 import Mx8Matrix, mx8_linear, mx8_linear_backward, mx8_product
    x, w, ids = torch.zeros(4, 32).bfloat16(), torch.zeros(32).bfloat16(), torch.zeros(4, dtype=torch.int64)
    m8, m4, spec = Mx8Matrix(4, 32, device="cpu"), Mx4Matrix(4, 32, device="cpu"), Z.dropout_spec(0.1, 1)
    with forward_ad.dual_level():
        d, v = forward_ad.make_dual(x, torch.ones_like(x)), forward_ad.make_dual(w, torch.ones_like(w))
        o = forward_ad.make_dual(torch.zeros(4, 4).bfloat16(), torch.zeros(4, 4).bfloat16())
        calls = [lambda d, v, o: L.embedding(ids, d), lambda d, v, o: L.embedding(ids, x, out=d), lambda d, v, o: L.embedding_backward(d, ids, x),
                 lambda d, v, o: L.embedding_backward(x, ids, d), lambda d, v, o: L.dropout(d, spec), lambda d, v, o: L.dropout(x, spec, out=d),
                 lambda d, v, o: L.rms_norm(d, w), lambda d, v, o: L.rms_norm(x, v), lambda d, v, o: L.rms_norm(x, w, residual=d),
                 lambda d, v, o: L.rms_norm_backward(d, x, w), lambda d, v, o: L.rms_norm_backward(x, d, w),
                 lambda d, v, o: L.rms_norm_backward(x, x, v), lambda d, v, o: L.rms_norm_backward(x, x, w, dh_in=d),
                 lambda d, v, o: L.rms_norm_backward(x, x, w, dweight=v),
                 lambda d, v, o: Mx8Matrix.of(d), lambda d, v, o: m8.fill(d), lambda d, v, o: mx8_linear(d, m8), lambda d, v, o: mx8_linear(d, m8, scratch=m8),
                 lambda d, v, o: mx8_linear(m8, m8, out=o), lambda d, v, o: mx8_product(m8, m8, out=o), lambda d, v, o: mx8_linear_backward(d, x, m8),
                 lambda d, v, o: Mx4Matrix.of(d, True), lambda d, v, o: mx4_linear(d, m4), lambda d, v, o: mx4_product(m4, m4, out=o),
                 lambda d, v, o: mx4_linear_backward(d, x, m4)]
        for call in calls:
            for mode in (torch.enable_grad, torch.no_grad):
                with mode():
                    refused(Z, "tangent", call, d, v, o)
                    refused(Z, "GPU", call, d.detach(), v.detach(), o.detach())
    for call in calls:
        refused(Z, "GPU", call, x, w, torch.zeros(4, 4).bfloat16())

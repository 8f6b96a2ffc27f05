"""Host-only checks of the matrix operators (no GPU): sizes, refusals before
any CUDA call, and the references themselves against small cases by hand."""

import numpy as np
import pytest
import torch

from _matrix_ref import mx4_decode, mx4_encode, mx4_pack, mx4_tile, newton_schulz


@pytest.fixture(scope="module")
def Z():
    from zero_partitioned_mixed_gb300.build import build_library
    build_library()
    import zero_partitioned_mixed_gb300 as Z
    return Z


def test_sizes(Z):
    assert Z.zero_mx4_codes_bytes(3, 33) == 3 * 32
    assert Z.zero_mx4_scales_bytes(129, 129) == 4 * 512
    assert Z.zero_mx4_scales_bytes(0, 10) == 0 and Z.zero_mx4_codes_bytes(10, 0) == 0
    assert Z.zero_mx4_codes_bytes((1 << 30) + 1, 1) == 0
    # two copies of X, three square matrices, and the norms
    need = Z.zero_orthogonalize_workspace_bytes(2, 100, 200)
    assert need >= 2 * (2 * 100 * 200 * 2 + 3 * 100 * 104 * 2)
    assert Z.zero_orthogonalize_workspace_bytes(0, 4, 4) == 0 and Z.zero_orthogonalize_workspace_bytes(1, 0, 4) == 0


@pytest.mark.parametrize("rows,cols", [(20, 30), (30, 9000), (300, 200)])
@pytest.mark.parametrize("src,dst", [(None, 256), (257, 256), (256, None), (256, 3)])
def test_matrices_are_checked_before_any_cuda_call(Z, rows, cols, src, dst):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_orthogonalize(1, rows, cols, [256, src], [256, dst], None, stream=0)
    assert e.value.code == 1 and "2-byte aligned" in str(e.value)


def test_refusals_come_before_any_cuda_call(Z):
    for call in (lambda: Z.zero_orthogonalize(7, 4, 4, [], [], None, stream=0),
                 lambda: Z.zero_orthogonalize(0, 4, 4, [16], [16], None, steps=0, stream=0),
                 lambda: Z.zero_mx4_quantize(1, 4, 32, 16, None, 16, stream=0),
                 lambda: Z.zero_mx4_matmul(9, 4, 4, 32, 16, 16, 16, 16, 16, stream=0),
                 lambda: Z.zero_muon_momentum(0, 8, [16] * 65, 32, 32, Z.muon_hyper(), 16, stream=0),
                 lambda: Z.zero_muon_apply(0, 8, 16, 16, [8], Z.muon_hyper(), 16, stream=0)):
        with pytest.raises(Z.ZeroError) as e:
            call()
        assert e.value.code == 1


def test_muon_state_has_the_header_s_size(Z):
    import ctypes
    assert ctypes.sizeof(Z._binding.MuonState) == 64 and ctypes.sizeof(Z._binding.MuonHyper) == 16


def test_newton_schulz_reference_on_a_diagonal():
    # on a diagonal matrix the iteration acts on each value by itself
    d = torch.tensor([3.0, 1.0, 0.5, 0.0], dtype=torch.float64)
    x = d / torch.linalg.vector_norm(d)
    for _ in range(5):
        x = 3.4445 * x - 4.7750 * x ** 3 + 2.0315 * x ** 5
    assert torch.allclose(newton_schulz(torch.diag(d)), torch.diag(x), atol=1e-14)
    tall = torch.randn(9, 4, dtype=torch.float64)
    assert torch.allclose(newton_schulz(tall), newton_schulz(tall.t()).t(), atol=1e-12)


def test_mx4_reference_by_hand():
    x = np.zeros((1, 33))
    x[0, :6] = [7.0, -5.0, 3.5, 2.5, 0.25, -0.75]      # largest exponent 2: scale 1
    x[0, 32] = 0.375                                   # 1.5 * 2^-2: scale 2^-4, code of 6
    codes, scales = mx4_encode(x)
    assert scales.tolist() == [[127, 123]]
    assert codes[0, :7].tolist() == [7, 14, 6, 4, 0, 10, 0] and codes[0, 32] == 7
    assert mx4_decode(codes, scales, 33)[0, [0, 1, 2, 3, 4, 5, 32]].tolist() == [6.0, -4.0, 4.0, 2.0, 0.0, -1.0, 0.375]
    assert mx4_pack(codes)[0, :3].tolist() == [7 | 14 << 4, 6 | 4 << 4, 0 | 10 << 4]
    t = mx4_tile(np.arange(1, 131, dtype=np.uint8)[:, None])
    assert t.size == 1024 and t[0] == 1 and t[16] == 2 and t[4] == 33 and t[512] == 129


@pytest.mark.parametrize("t", [torch.zeros(64).expand(100, 64), torch.zeros(100, 1).expand(100, 64),
                               torch.zeros(200).as_strided((100, 64), (1, 1)), torch.zeros(1).expand(7, 1)],
                         ids=["one row for all", "one column for all", "overlapping rows", "one value for all"])
def test_rows_that_share_memory_are_refused(Z, t):
    # a row stride below the width: the rows do not lie one after the other, as the calls read and write them
    from zero_partitioned_mixed_gb300 import mx4
    with pytest.raises(Z.ZeroError) as e:
        mx4._rows(t)
    assert e.value.code == 1 and "contiguous rows" in str(e.value)


def test_leading_dimensions_of_ordinary_tensors(Z):
    from zero_partitioned_mixed_gb300 import mx4
    room = torch.zeros(4096)
    for shape, stride, ld in (((5, 7), (7, 1), 7), ((5, 7), (9, 1), 9), ((1, 7), (0, 1), 7), ((1, 7), (3, 1), 7),
                              ((5, 1), (1, 1), 1), ((5, 1), (4, 3), 4), ((0, 7), (0, 1), 7), ((5, 0), (0, 1), 0),
                              ((5, 0), (1, 1), 1)):
        assert mx4._rows(room.as_strided(shape, stride)) == ld, (shape, stride)


def test_tensors_in_host_memory_are_refused(Z):
    from zero_partitioned_mixed_gb300 import mx4
    x, m = torch.zeros(4, 32, dtype=torch.bfloat16), mx4.Mx4Matrix(4, 32, device="cpu")
    for call in (lambda: mx4.Mx4Matrix.of(x), lambda: mx4.Mx4Matrix.of(x, transpose=True), lambda: m.fill(x), m.values,
                 lambda: mx4.mx4_product(m, m), lambda: mx4.mx4_product(m, m, out=torch.zeros(4, 4, dtype=torch.bfloat16)),
                 lambda: mx4.mx4_linear(x, m), lambda: mx4.mx4_linear_backward(x, x, m)):
        with pytest.raises(Z.ZeroError) as e:
            call()
        assert e.value.code == 1 and "GPU" in str(e.value)


@pytest.mark.parametrize("state", [260, 257])
def test_a_step_s_orthogonalisation_checks_its_state(Z, state):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_orthogonalize(1, 20, 30, [256], [256], None, stream=0, state=state)
    assert e.value.code == 1 and "state" in str(e.value)


def test_shared_memory_that_is_read_in_wider_pieces_is_aligned_for_them():
    import pathlib
    import re
    csrc = pathlib.Path(__file__).resolve().parents[1] / "zero_partitioned_mixed_gb300" / "csrc"
    found = 0
    for path in sorted(csrc.glob("*.cu*")):
        t = path.read_text()
        for align, name in re.findall(r"__shared__ (__align__\(\d+\) )?(?:uint8_t|unsigned char|uint16_t|__half) (\w+)\[", t):
            casts = re.findall(rf"reinterpret_cast<(?:const )?(uint\d_t|uint32_t|uint64_t|uint2|uint4|float4) ?\*>\([^;]*?\b{name}\b", t)
            if casts:
                found += 1
                assert align, f"{path.name}: {name} is read as {casts[0]}"
    assert found >= 1


def test_a_linear_layer_refuses_to_drop_its_input_s_gradient(Z):
    # the call makes no autograd graph: without a word, whatever made x would train on no gradient
    from zero_partitioned_mixed_gb300 import mx4
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16, requires_grad=True), mx4.Mx4Matrix(8, 32, device="cpu")
    with pytest.raises(Z.ZeroError) as e:
        mx4.mx4_linear(x, w)
    assert e.value.code == 1 and "mx4_linear_backward" in str(e.value)
    for quiet in (lambda: mx4.mx4_linear(x.detach(), w), torch.no_grad()(lambda: mx4.mx4_linear(x, w))):
        with pytest.raises(Z.ZeroError) as e:
            quiet()
        assert "GPU" in str(e.value)      # as far as a host tensor gets

"""Sizes past the library's bounds, where products of sizes no longer fit 64 bits:
the queries of the quantised rows and the MXFP4 product return 0, and the binding
refuses them before it compares a buffer with a size that wrapped round."""
import pytest

torch = pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import _lib as ops  # noqa: E402

BIG = 1 << 62


def test_size_queries_of_impossible_sizes():
    L = ops.lib()
    assert L.w4a4_mx4_scale_stride((1 << 24) + 32) == 0 and L.w4a4_mx4_scale_stride(1 << 24) == 1 << 19
    for n, k in ((BIG, 64), ((1 << 26) + 1, 32), (32, (1 << 24) + 32), (32, BIG)):
        assert L.w4a4_mx4_packed_bytes(n, k) == 0
    assert L.w4a4_mx4_packed_bytes(1 << 26, 256) == (1 << 21) * 2 * 2176
    for fmt in range(5):
        for m, k in ((BIG, 64), ((1 << 26) + 1, 32), (4, (1 << 24) + 32), (4, BIG)):
            assert L.w4a4_act_format_code_bytes(fmt, m, k) == 0
            assert L.w4a4_act_format_scale_bytes(fmt, m, k) == 0
            assert L.w4a4_act_format_operand_bytes(fmt, m, k) == 0
    assert L.w4a4_act_format_code_bytes(2, 1 << 26, 1 << 24) == 1 << 50


def test_binding_refuses_impossible_sizes():
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 8), dtype=torch.uint8)
    x = torch.zeros((4, 64))
    for n, k, match in ((BIG, 64, "n = .*at most"), ((1 << 26) + 1, 64, "n = .*at most"), (4, BIG, "k = .*at most"), (-1, 64, "negative")):
        with pytest.raises(ops.W4A4Error, match=match):
            ops.repack_mx4(codes.reshape(-1), scales.reshape(-1), n, k, out=torch.zeros(1, dtype=torch.uint8))
        with pytest.raises(ops.W4A4Error, match=match):
            ops.gemm_mx4(codes, codes, scales, n, k)
    with pytest.raises(ops.W4A4Error, match="k = .*at most"):
        ops.dequantize_act(codes, scales, BIG, ops.ACT_MX4)
    with pytest.raises(ops.W4A4Error, match="k = .*at most"):
        ops.quantize_mx4(x, k=BIG)
    with pytest.raises(ops.W4A4Error, match="k = .*at most"):
        ops.glu_quantize(x, x, ops.ACT_INT8, k=BIG)

"""Refusals of the quantised-row producers, the read-back and the MXFP4
product, on the CPU: the C ABI's statuses (fake device pointers are never
dereferenced) and the binding's checks."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import _lib as ops  # noqa: E402

OK, INVALID, KMUL, MISALIGNED, DTYPE, WS, HIP = range(7)
F32, F16, BF16 = 0, 1, 2
A, B, C = 0x10000000, 0x20000000, 0x30000000
GPU_ONLY = "must live on the GPU"


def P(x):
    return ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def L():
    return ops.lib()


def test_size_queries(L):
    assert [L.w4a4_mx4_scale_stride(k) for k in (0, 32, 256, 288, 5120, 17408, 33, -32)] == [0, 8, 8, 16, 160, 544, 0, 0]
    assert L.w4a4_mx4_packed_bytes(17408, 5120) == 544 * 20 * 4352
    assert L.w4a4_mx4_packed_bytes(33, 288) == 2 * 2 * 4352
    assert L.w4a4_mx4_packed_bytes(8, 40) == 0
    for fmt, codes, scales, operand in [(0, 20 * 32, 20 * 8, L.w4a4_act_operand_bytes(20, 64)), (1, 20 * 32, 20 * 8, 0),
                                        (2, 20 * 64, 20 * 8, L.w4a4_act8_operand_bytes(20, 64)), (3, 20 * 32, 20 * 8, 0),
                                        (4, 20 * 32, 20 * 8, 0), (5, 0, 0, 0), (-1, 0, 0, 0)]:
        assert L.w4a4_act_format_code_bytes(fmt, 20, 64) == codes
        assert L.w4a4_act_format_scale_bytes(fmt, 20, 64) == scales
        assert L.w4a4_act_format_operand_bytes(fmt, 20, 64) == operand
    assert L.w4a4_act_format_scale_bytes(0, 20, 96) == 20 * 3 * 4
    assert L.w4a4_act_format_operand_bytes(1, 16, 64) == L.w4a4_small_act_operand_bytes(16, 64)
    assert L.w4a4_act_format_code_bytes(0, 20, 48) == 0
    assert L.w4a4_gemm_mx4_workspace_bytes(-1, 1, 32) == 0 and L.w4a4_gemm_mx4_workspace_bytes(1, 1, 33) == 0


def test_quantize_mx4_statuses(L):
    f = L.w4a4_quantize_mx4
    assert f(P(A), 3, 4, 64, 64, 1, P(A), P(A), None) == DTYPE
    assert f(P(A), F32, -1, 64, 64, 1, P(A), P(A), None) == INVALID
    assert f(P(A), F32, 4, 64, 63, 1, P(A), P(A), None) == INVALID
    assert f(P(A), F32, 4, 1 << 25, 1 << 25, 1, P(A), P(A), None) == INVALID
    assert f(P(A), F32, 1 << 26, 1 << 20, 1 << 20, 1, P(A), P(A), None) == INVALID  # past 2^32 threads
    assert f(P(A), F32, 4, 48, 48, 1, P(A), P(A), None) == KMUL
    assert f(None, F32, 4, 64, 64, 1, P(A), P(A), None) == INVALID
    assert f(P(A), F32, 4, 64, 64, 1, None, P(A), None) == INVALID
    assert f(P(A), F32, 4, 64, 64, 1, P(A), None, None) == INVALID
    assert f(P(A + 2), F32, 4, 64, 64, 1, P(A), P(A), None) == MISALIGNED
    assert f(P(A + 1), BF16, 4, 64, 64, 1, P(A), P(A), None) == MISALIGNED
    assert f(P(A), F32, 4, 64, 64, 1, P(A + 8), P(A), None) == MISALIGNED
    assert f(P(A), F32, 4, 64, 64, 1, P(A), P(A + 4), None) == MISALIGNED
    assert f(None, F32, 0, 64, 64, 1, None, None, None) == OK and f(None, F32, 4, 0, 0, 1, None, None, None) == OK


def test_dequantize_act_statuses(L):
    f = L.w4a4_dequantize_act
    assert f(5, P(A), P(A), 4, 64, P(A), F32, 64, None) == INVALID
    assert f(0, P(A), P(A), 4, 64, P(A), 9, 64, None) == DTYPE
    assert f(0, P(A), P(A), 4, 64, P(A), F32, 63, None) == INVALID
    assert f(0, P(A), P(A), 4, 33, P(A), F32, 64, None) == KMUL
    for bad in range(3):
        args = [P(A), P(A), P(A)]
        args[bad] = None
        assert f(0, args[0], args[1], 4, 64, args[2], F32, 64, None) == INVALID
    assert f(0, P(A + 8), P(A), 4, 64, P(A), F32, 64, None) == MISALIGNED
    assert f(3, P(A), P(A + 4), 4, 64, P(A), F32, 64, None) == MISALIGNED
    assert f(0, P(A), P(A), 4, 64, P(A + 2), F32, 64, None) == MISALIGNED
    assert f(0, None, None, 0, 64, None, F32, 64, None) == OK


def norm(L, x=A, xdt=F32, ldx=64, res=None, rdt=F16, ldr=64, w=A, eps=1e-6, m=4, k=64, h=None, ldh=64, fmt=0, codes=B,
         scales=B, operand=None, nbytes=0):
    return L.w4a4_rms_norm_quantize(P(x), xdt, ldx, P(res), rdt, ldr, P(w), eps, m, k, P(h), ldh, fmt, P(codes), P(scales),
                                    P(operand), nbytes, None)


def test_norm_statuses(L):
    assert norm(L, xdt=3) == DTYPE and norm(L, rdt=-1) == DTYPE
    for bad in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(L, eps=bad) == INVALID
    assert norm(L, fmt=5) == INVALID and norm(L, m=-1) == INVALID and norm(L, ldx=63) == INVALID
    assert norm(L, res=B, ldr=63) == INVALID and norm(L, h=C, ldh=63) == INVALID
    assert norm(L, k=65536 * 512, ldx=65536 * 512) == INVALID and norm(L, m=65535 * 32 + 1) == INVALID
    assert norm(L, k=40) == KMUL
    assert norm(L, x=None) == INVALID and norm(L, codes=None) == INVALID and norm(L, scales=None) == INVALID
    assert norm(L, fmt=3, operand=C, nbytes=1 << 20) == INVALID  # MXFP4 has no operand
    assert norm(L, fmt=1) == INVALID and norm(L, fmt=1, m=17, operand=C, nbytes=1 << 20) == INVALID
    # in place: h is x only when the types and strides are equal, the residual when the strides are
    assert norm(L, h=A) == INVALID and norm(L, h=A, rdt=F32, ldh=72) == INVALID
    assert norm(L, res=C, h=C, ldr=64, ldh=72) == INVALID
    assert norm(L, x=A + 2) == MISALIGNED and norm(L, res=C + 1) == MISALIGNED and norm(L, h=C + 1) == MISALIGNED
    assert norm(L, w=A + 2) == MISALIGNED and norm(L, codes=B + 8) == MISALIGNED and norm(L, scales=B + 2) == MISALIGNED
    assert norm(L, fmt=3, scales=B + 4) == MISALIGNED and norm(L, operand=C + 16, nbytes=1 << 20) == MISALIGNED
    for fmt, m in ((0, 4), (1, 4), (2, 4)):
        need = L.w4a4_act_format_operand_bytes(fmt, m, 64)
        assert need > 0 and norm(L, fmt=fmt, m=m, operand=C, nbytes=need - 1) == WS
    assert norm(L, m=0, x=None, codes=None, scales=None) == OK
    assert norm(L, k=0, ldx=0, x=None, codes=None, scales=None) == OK


def glu(L, gate=A, up=C, dt=F32, m=4, k=64, ldg=64, ldu=64, act=0, fmt=0, codes=B, scales=B, operand=None, nbytes=0):
    return L.w4a4_glu_quantize(P(gate), P(up), dt, m, k, ldg, ldu, act, fmt, P(codes), P(scales), P(operand), nbytes, None)


def test_glu_statuses(L):
    assert glu(L, dt=3) == DTYPE and glu(L, act=2) == INVALID and glu(L, fmt=-1) == INVALID
    assert glu(L, ldg=63) == INVALID and glu(L, ldu=63) == INVALID and glu(L, m=-1) == INVALID
    assert glu(L, k=40) == KMUL
    assert glu(L, gate=None) == INVALID and glu(L, up=None) == INVALID and glu(L, codes=None) == INVALID
    assert glu(L, gate=A + 2) == MISALIGNED and glu(L, up=C + 2) == MISALIGNED and glu(L, codes=B + 4) == MISALIGNED
    assert glu(L, fmt=4, operand=C, nbytes=1 << 20) == INVALID and glu(L, fmt=1, m=17, operand=C, nbytes=1 << 20) == INVALID
    assert glu(L, fmt=2, operand=C, nbytes=1) == WS
    assert glu(L, m=0, gate=None, up=None, codes=None, scales=None) == OK


def test_mx4_product_statuses(L):
    f = L.w4a4_gemm_mx4
    assert f(P(A), P(A), P(A), P(A), 3, 4, 64, 64, 64, None, 0, None) == DTYPE
    assert f(P(A), P(A), P(A), P(A), F32, -4, 64, 64, 64, None, 0, None) == INVALID
    assert f(P(A), P(A), P(A), P(A), F32, 4, 64, 64, 63, None, 0, None) == INVALID
    assert f(P(A), P(A), P(A), P(A), F32, 65535 * 32 + 1, 64, 64, 64, None, 0, None) == INVALID
    assert f(P(A), P(A), P(A), P(A), F32, 4, 64, 48, 64, None, 0, None) == KMUL
    for bad in range(4):
        args = [P(A)] * 4
        args[bad] = None
        assert f(*args, F32, 4, 64, 64, 64, None, 0, None) == INVALID
    assert f(P(A + 8), P(A), P(A), P(A), F32, 4, 64, 64, 64, None, 0, None) == MISALIGNED
    assert f(P(A), P(A + 8), P(A), P(A), F32, 4, 64, 64, 64, None, 0, None) == MISALIGNED
    assert f(P(A), P(A), P(A + 4), P(A), F32, 4, 64, 64, 64, None, 0, None) == MISALIGNED
    assert f(P(A), P(A), P(A), P(A + 2), F32, 4, 64, 64, 64, None, 0, None) == MISALIGNED
    assert f(P(A), P(A), P(A), P(A + 1), BF16, 4, 64, 64, 64, None, 0, None) == MISALIGNED
    assert f(None, None, None, None, F32, 0, 64, 64, 64, None, 0, None) == OK
    assert f(None, None, None, None, F32, 4, 0, 64, 0, None, 0, None) == OK
    r = L.w4a4_repack_mx4
    assert r(P(A), P(A), 4, 48, P(A), None) == KMUL and r(P(A), P(A), -4, 64, P(A), None) == INVALID
    assert r(None, P(A), 4, 64, P(A), None) == INVALID and r(P(A), P(A), 4, 64, None, None) == INVALID
    assert r(P(A + 8), P(A), 4, 64, P(A), None) == MISALIGNED and r(P(A), P(A + 4), 4, 64, P(A), None) == MISALIGNED
    assert r(P(A), P(A), 4, 64, P(A + 8), None) == MISALIGNED
    assert r(None, None, 0, 64, None, None) == OK


# ---------------------------------------------------------------- binding

def raises(match, fn, *a, **kw):
    with pytest.raises(ops.W4A4Error, match=match):
        fn(*a, **kw)


M, N, K = 20, 70, 96


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def u8(*shape):
    return zeros(*shape, dtype=torch.uint8)


def test_well_formed_host_tensors_reach_the_device_check():
    x = zeros(M, K, dtype=torch.bfloat16)
    raises(GPU_ONLY, ops.quantize_mx4, x)
    raises(GPU_ONLY, ops.quantize_mx4, zeros(M, K + 5), k=K)
    raises(GPU_ONLY, ops.dequantize_act, u8(M, K // 2), u8(M, 8), K, ops.ACT_MX4)
    raises(GPU_ONLY, ops.rms_norm_quantize, x, zeros(K), 1e-6, ops.ACT_INT8, residual=x)
    raises(GPU_ONLY, ops.glu_quantize, x, x, ops.ACT_MX4_H32)
    raises(GPU_ONLY, ops.gemm_mx4, u8(ops.mx4_packed_bytes(N, K)), u8(M, K // 2), u8(M, 8), N, K)
    raises(GPU_ONLY, ops.repack_mx4, u8(N, K // 2), u8(N, 8), N, K)


def test_binding_refuses_wrong_types_shapes_and_strides():
    x = zeros(M, K)
    raises("x: dtype", ops.quantize_mx4, x.double())
    raises("x: strides", ops.quantize_mx4, zeros(K, M + 12).t()[:, :K])
    raises("not a multiple of 32", ops.quantize_mx4, zeros(M, 40))
    raises("codes: .* bytes", ops.quantize_mx4, x, codes=u8(M * K // 2 - 1))
    raises("scales: .* bytes", ops.quantize_mx4, x, scales=u8(M * 8 - 1))
    raises("scales: dtype", ops.quantize_mx4, x, scales=zeros(M, 8))
    raises("unknown format", ops.dequantize_act, u8(M, K // 2), u8(M, 8), K, 7)
    raises("codes: dtype", ops.dequantize_act, u8(M, K), zeros(M, K // 32), K, ops.ACT_INT8)
    raises("out: shape", ops.dequantize_act, u8(M, K // 2), u8(M, 8), K, ops.ACT_MX4, out=zeros(M, K - 1))
    raises("dtype: dtype", ops.dequantize_act, u8(M, K // 2), u8(M, 8), K, ops.ACT_MX4, dtype=torch.float64)


def test_binding_norm_and_glu_checks():
    x, r, w = zeros(M, K), zeros(M, K, dtype=torch.float16), zeros(K)
    n = ops.rms_norm_quantize
    raises("weight: dtype", n, x, w.half(), 1e-6, ops.ACT_MX4)
    raises("weight: .* bytes", n, x, zeros(K - 1), 1e-6, ops.ACT_MX4)
    raises("eps", n, x, w, 0.0, ops.ACT_MX4)
    raises("eps", n, x, w, float("nan"), ops.ACT_MX4)
    raises("residual: shape", n, x, w, 1e-6, ops.ACT_MX4, residual=r[: M - 1])
    raises("h: dtype", n, x, w, 1e-6, ops.ACT_MX4, residual=r, h=x)
    raises("h: shape", n, x, w, 1e-6, ops.ACT_MX4, h=zeros(M, K - 32))
    raises("unknown format", n, x, w, 1e-6, 9)
    raises("at most 16", n, x, w, 1e-6, ops.ACT_INT4_SMALL)
    raises("MXFP4 rows have none", n, x, w, 1e-6, ops.ACT_MX4, operand=u8(1 << 16))
    raises("operand: .* bytes", n, x, w, 1e-6, ops.ACT_INT8, operand=u8(8))
    g = ops.glu_quantize
    raises("up: dtype", g, x, r, ops.ACT_INT4)
    raises("up: shape", g, x, zeros(M - 1, K), ops.ACT_INT4)
    raises("unknown activation", g, x, x, ops.ACT_INT4, act=2)
    raises("codes: dtype", g, x, x, ops.ACT_INT8, codes=u8(M, K))
    raises("at most 16", g, x, x, ops.ACT_INT4_SMALL)


def test_binding_product_checks():
    packed, c, s = u8(ops.mx4_packed_bytes(N, K)), u8(M, K // 2), u8(M, 8)
    raises("packed: .* bytes", ops.gemm_mx4, packed[:-1], c, s, N, K)
    raises("codes: .* bytes", ops.gemm_mx4, u8(ops.mx4_packed_bytes(N, 2 * K)), c, u8(M, 16), N, 2 * K)
    raises("scales: .* bytes", ops.gemm_mx4, packed, c, u8(M, 7), N, K)
    raises("y: shape", ops.gemm_mx4, packed, c, s, N, K, y=zeros(M, N - 1))
    raises("y: dtype", ops.gemm_mx4, packed, c, s, N, K, y=zeros(M, N, dtype=torch.float64))
    raises("codes must be", ops.gemm_mx4, packed, c, s, N, 40)
    raises("codes: .* bytes", ops.repack_mx4, u8(N, K // 2 - 1), u8(N, 8), N, K)
    raises("out: .* bytes", ops.repack_mx4, u8(N, K // 2), u8(N, 8), N, K, out=packed[:-1])


def test_binding_refuses_rows_of_another_width():
    """Buffers large enough, but rows of another k's width."""
    c, s = u8(M, K), u8(M, 8)
    raises("codes: rows of 96, expected 48", ops.dequantize_act, c, s, K, ops.ACT_MX4)
    raises("scales: rows of 16, expected 8", ops.dequantize_act, u8(M, K // 2), u8(M, 16), K, ops.ACT_MX4)
    raises("scales: rows of 4, expected 3", ops.dequantize_act, zeros(M, K, dtype=torch.int8), zeros(M, 4), K, ops.ACT_INT8)
    packed = u8(ops.mx4_packed_bytes(N, K))
    raises("codes: rows of 96", ops.gemm_mx4, packed, c, s, N, K)
    raises("scales: rows of 16", ops.gemm_mx4, packed, u8(M, K // 2), u8(M, 16), N, K)
    raises("codes: rows of 96", ops.repack_mx4, u8(N, K), u8(N, 8), N, K)
    raises("codes: rows of 96", ops.quantize_mx4, zeros(M, K), codes=c)
    raises("scales: rows of 16", ops.glu_quantize, zeros(M, K), zeros(M, K), ops.ACT_MX4, scales=u8(M, 16))
    raises(GPU_ONLY, ops.quantize_mx4, zeros(M, K), codes=u8(M * K), scales=u8(M + 3, 8))  # larger buffers are fine


def test_mx4_product_workspace(L):
    """The rows as records, and the partial sums where K is split; nothing for
    the streamed sizes."""
    size = L.w4a4_gemm_mx4_workspace_bytes
    assert size(32, 17408, 5120) == 0 and size(64, 8192, 512) == 0 and size(0, 64, 64) == 0 and size(64, 0, 64) == 0
    assert size(-1, 64, 64) == 0 and size(64, 64, 48) == 0 and size(64, 64, 0) == 0
    rows = L.w4a4_mx4_packed_bytes(302, 64)
    assert size(302, 10240, 64) == (rows + 255) // 256 * 256
    split = size(65, 5120, 17408) - (L.w4a4_mx4_packed_bytes(65, 17408) + 255) // 256 * 256
    assert split > 0 and split % (65 * 5120 * 4) == 0
    f, need = L.w4a4_gemm_mx4, size(302, 10240, 64)
    args = [P(A), P(A), P(A), P(A), F32, 302, 10240, 64, 10240]
    assert f(*args, None, need, None) == INVALID
    assert f(*args, P(A + 16), need, None) == MISALIGNED
    assert f(*args, P(A), need - 1, None) == WS

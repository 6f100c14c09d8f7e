"""Infinities and NaN in quantised rows: what reaches a block, and what does not.

The producers' codes and scales are compared for equality with a plain form
written here; a block whose values are not all finite must not read back as
finite numbers, and no other block may change."""
import numpy as np
import pytest

import rows_twin as twin

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FORMATS = {"int4": 0, "int4_small": 1, "int8": 2, "mx4": 3, "mx4_h32": 4}
INF, NAN = np.float32(np.inf), np.float32(np.nan)


@pytest.fixture(scope="module")
def ops():
    from hadamard_rotated_w4a4_amd import _lib
    _lib.lib()
    return _lib


def say(msg):
    print(f"[gpu nonfinite] {msg}", flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def int_rows(v, top, rotate, nan_scale):
    """Blocks on the int4 or int8 grid, non-finite values included: a NaN product
    of value and inverse scale takes code -top, unless the block is a zero
    block.  nan_scale: a NaN among the block's values makes its scale NaN
    (and zero codes); otherwise the maximum ignores it."""
    with np.errstate(all="ignore"):
        b = v.reshape(v.shape[0], -1, 32)
        u = twin.butterflies(b) if rotate else b
        a = np.abs(u)
        amax = a.max(-1) if nan_scale else np.where(np.isnan(a), np.float32(0), a).max(-1)
        d = amax / np.float32(top)
        live = d >= np.float32(1.17549435e-38)
        inv = np.where(live, np.float32(1) / np.where(live, d, np.float32(1)), np.float32(0)).astype(np.float32)
        t = u * inv[..., None]
        q = np.copysign(np.floor(np.abs(t.astype(np.float64)) + 0.5), t)
        q = np.where(np.isnan(t), -top, np.clip(q, -top, top))
        q = np.where(live[..., None], q, 0).astype(np.int8)
        s = np.where(live, d * twin.C32 if rotate else d, np.where(np.isnan(d), d, np.float32(0)))
    return q.reshape(v.shape), s.astype(np.float32)


def check(fmt, codes, scales, v):
    torch.cuda.synchronize()
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    if fmt.startswith("mx4"):
        wc, ws = twin.mx4_rows(v, fmt == "mx4_h32")
    else:
        wc, ws = int_rows(v, 127 if fmt == "int8" else 7, True, True)
        wc = twin.int4_bytes(wc) if fmt.startswith("int4") else wc
    assert np.array_equal(s.reshape(ws.shape), ws, equal_nan=True), f"scales {s.reshape(ws.shape)[:, :6]}, expected {ws[:, :6]}"
    assert np.array_equal(c.reshape(wc.shape), wc)


def reads_non_finite(ops, fmt, codes, scales, k, blocks):
    """Exactly the given (row, block) pairs read back as no finite number."""
    f = ops.ACT_MX4 if fmt == "mx4" else FORMATS[fmt]
    y = ops.dequantize_act(codes, scales, k, f).cpu().numpy().reshape(codes.shape[0], -1, 32)
    lost = ~np.isfinite(y)
    want = np.zeros(lost.shape[:2], bool)
    for r, b in blocks:
        want[r, b] = True
    assert np.array_equal(lost.any(-1), want) and np.array_equal(lost.all(-1), want)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("k", [96, 5120, 8224, 32800])  # one, two and four pieces a thread, and rows walked twice
def test_norm_of_a_row_that_overflows(ops, fmt, k):
    """Finite inputs whose fp16 sum is infinite: the root is 0, the infinity's
    own block is lost, the row's others are zero; other rows are untouched."""
    say(f"rms_norm_quantize {fmt} k={k}")
    rng = np.random.default_rng(k)
    m = 4
    x = rng.standard_normal((m, k)).astype(np.float32)
    r = rng.standard_normal((m, k)).astype(np.float16)
    x[1, 33], r[1, 33] = 60000, 60000
    x[2, 64], r[2, 64] = -60000, -60000
    w = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    with np.errstate(all="ignore"):
        hn, v = twin.norm(x, r.astype(np.float32), torch.float16, w, 1e-6)
    assert np.isinf(hn[1, 33]) and np.isinf(hn[2, 64]) and np.isfinite(hn[[0, 3]]).all()
    both = torch.zeros(ops.act_format_operand_bytes(FORMATS[fmt], m, k), dtype=torch.uint8, device="cuda")
    for operand in ([both] if fmt == "int4_small" else [None] if fmt.startswith("mx4") else [None, both]):
        codes, scales, h = ops.rms_norm_quantize(dev(x), dev(w), 1e-6, FORMATS[fmt], residual=dev(r), operand=operand)
        assert np.array_equal(h.float().cpu().numpy(), hn)
        check(fmt, codes, scales, v)
        reads_non_finite(ops, fmt, codes, scales, k, [(1, 1), (2, 2)])


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_norm_of_a_row_with_a_nan(ops, fmt):
    say(f"rms_norm_quantize NaN {fmt}")
    k = 160
    x = np.random.default_rng(2).standard_normal((3, k)).astype(np.float32)
    x[1, 7] = NAN
    with np.errstate(all="ignore"):
        _, v = twin.norm(x, None, torch.float32, None, 1e-6)
    operand = torch.zeros(ops.act_format_operand_bytes(1, 3, k), dtype=torch.uint8, device="cuda") if fmt == "int4_small" else None
    codes, scales, _ = ops.rms_norm_quantize(dev(x), None, 1e-6, FORMATS[fmt], operand=operand)
    check(fmt, codes, scales, v)
    reads_non_finite(ops, fmt, codes, scales, k, [(1, b) for b in range(5)])


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_glu_of_infinities_and_nan(ops, fmt, act):
    say(f"glu_quantize {fmt} {act}")
    m, k = 9, 128
    rng = np.random.default_rng(3)
    g, u = (rng.standard_normal((m, k)).astype(np.float32) for _ in range(2))
    g[0, 40], u[0, 40] = INF, 0.5       # infinite
    g[1, 40], u[1, 40] = 1.5, -INF
    g[2, 0], u[2, 0] = 3e38, 3e38       # overflows in the one rounding to fp32
    g[3, 70], u[3, 70] = INF, 0.0       # NaN
    g[4, 70], u[4, 70] = 0.0, INF
    g[5, 127] = NAN
    u[6, 127] = NAN
    g[7, 3], g[7, 4], u[7, 3:5] = INF, INF, (1.0, -1.0)  # two of opposite signs
    with np.errstate(all="ignore"):
        v = twin.gated(g, u, getattr(twin, act))
    lost = [(0, 1), (1, 1), (2, 0), (3, 2), (4, 2), (5, 3), (6, 3), (7, 0)]
    operand = torch.zeros(ops.act_format_operand_bytes(1, m, k), dtype=torch.uint8, device="cuda") if fmt == "int4_small" else None
    a = ops.GLU_SILU if act == "silu" else ops.GLU_GELU_TANH
    codes, scales = ops.glu_quantize(dev(g), dev(u), FORMATS[fmt], act=a, operand=operand)
    check(fmt, codes, scales, v)
    reads_non_finite(ops, fmt, codes, scales, k, lost)
    # a gate of minus infinity: the formula has no value there
    g[8, 100] = -INF
    codes, scales = ops.glu_quantize(dev(g), dev(u), FORMATS[fmt], act=a, operand=operand)
    reads_non_finite(ops, fmt, codes, scales, k, lost + [(8, 3)])


@pytest.mark.parametrize("m", [5, 40])
def test_an_overflow_reaches_the_product_of_the_operand(ops, m):
    """Rows of a prepared product are lost with their block, and only those."""
    say(f"glu_quantize -> prepared products, m={m}")
    n, k = 64, 256
    rng = np.random.default_rng(m)
    g, u = (dev(rng.standard_normal((m, k)).astype(np.float32)) for _ in range(2))
    packed = ops.prepare_weights(dev((rng.standard_normal((n, k)) * 0.02).astype(np.float32)))

    def products():
        out = []
        for fmt in ([ops.ACT_INT4, ops.ACT_INT8] if m > 16 else [ops.ACT_INT4_SMALL]):
            operand = torch.zeros(ops.act_format_operand_bytes(fmt, m, k), dtype=torch.uint8, device="cuda")
            ops.glu_quantize(g, u, fmt, operand=operand)
            f = {ops.ACT_INT4: ops.gemm_prepared, ops.ACT_INT8: ops.gemm_a8_prepared, ops.ACT_INT4_SMALL: ops.gemm_prepared_small}[fmt]
            out.append(f(packed, operand, m, n, k).cpu().numpy())
        return out

    clean = products()
    g[2, 37], u[2, 37] = float("inf"), 1.0
    g[4, 200] = float("nan")
    for y, want in zip(products(), clean):
        hit = np.zeros(m, bool)
        hit[[2, 4]] = True
        assert not np.isfinite(y[hit]).any() and np.array_equal(y[~hit], want[~hit])


@pytest.mark.parametrize("m", [5, 40])
def test_an_overflow_reaches_the_products_of_codes_and_scales(ops, m):
    """As above for the products that read the public codes and scales, dense and
    per routed row."""
    say(f"glu_quantize -> products of codes and scales, m={m}")
    n, k, experts = 64, 256, 3
    rng = np.random.default_rng(m + 1)
    g, u = (dev(rng.standard_normal((m, k)).astype(np.float32)) for _ in range(2))
    packed = [ops.prepare_weights(dev((rng.standard_normal((n, k)) * 0.02).astype(np.float32))) for _ in range(experts)]
    ids = dev(rng.integers(0, experts, (m, 1)).astype(np.int32))

    def products():
        c4, s4 = ops.glu_quantize(g, u, ops.ACT_INT4)
        c8, s8 = ops.glu_quantize(g, u, ops.ACT_INT8)
        out = [ops.gemm(packed[0], c4, s4, n, k), ops.gemm_noalloc(packed[0], c4, s4, n, k), ops.gemm_a8(packed[0], c8, s8, n, k),
               ops.gemm_id(torch.cat(packed), experts, c4, s4, 1, ids, n, k).reshape(m, n)]
        return [y.cpu().numpy() for y in out]

    clean = products()
    g[2, 37], u[2, 37] = float("inf"), 1.0
    g[4, 200] = float("nan")
    hit = np.zeros(m, bool)
    hit[[2, 4]] = True
    for i, (y, want) in enumerate(zip(products(), clean)):
        assert not np.isfinite(y[hit]).any(), i
        assert np.array_equal(y[~hit], want[~hit]), i


@pytest.mark.parametrize("call,top,rotate", [("rotate_quantize_act", 7, True), ("rotate_quantize_act8", 127, True), ("quantize_act", 7, False)])
def test_quantisers_of_a_matrix_keep_their_codes(ops, call, top, rotate):
    """The quantisers of a matrix in memory: a product that is NaN (an infinite
    scale, or a NaN among unrotated values) has code -top, a block of NaN only
    is a zero block."""
    say(f"{call}")
    x = np.random.default_rng(5).standard_normal((6, 128)).astype(np.float32)
    x[0, 40], x[1, 33], x[2, 70] = INF, -INF, NAN
    x[3, 0:2] = INF, -INF
    x[4, 64:96] = NAN
    x[5, :32] = 3e38 * np.sign(x[5, :32])  # sums of both signs overflow in the rotation
    q, s = int_rows(x, top, rotate, False)
    codes, scales = getattr(ops, call)(dev(x))
    torch.cuda.synchronize()
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), q if top == 127 else twin.int4_bytes(q))


def test_int4_rounding_borders(ops):
    """Values on and one fp32 either side of every half and whole step, against
    an inverse scale of exactly 1: half away from zero."""
    say("quantize_act borders")
    edge = np.arange(0.5, 7.0, 0.5, dtype=np.float32)
    near = np.concatenate((edge, np.nextafter(edge, INF), np.nextafter(edge, -INF), [np.float32(1e-30), np.float32(0.0)])).astype(np.float32)
    near = np.insert(near, 31, 7.0)
    x = np.zeros((2, 64), np.float32)
    x[0, :near.size], x[1, :near.size] = near, -near
    x[:, 63] = 7.0
    q, s = int_rows(x, 7, False, False)
    assert (s == 1).all()
    codes, scales = ops.quantize_act(dev(x))
    torch.cuda.synchronize()
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), twin.int4_bytes(q))

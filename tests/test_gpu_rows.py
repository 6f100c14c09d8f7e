"""GPU tests of the quantised-row producers (MXFP4 quantiser, residual + RMS
norm, gated activation) and the read-back, against the plain implementations
of rows_twin.

The codes, scales and h are compared for equality: the definition fixes every
rounding, and what it leaves unordered (the sum of squares, the activation
function) is evaluated in fp64 on both sides, where two evaluations differ by
at most about 2^-40 and so round to the same fp32 value but for one case in
some 2^15 (a last-place difference that moves a code in one of those in 2^20).
Operand buffers are compared with what the quantisers write for the same
values.  Buffers are filled with a pattern first and have a margin after the
last row: every byte outside the outputs keeps it."""
import numpy as np
import pytest

import rows_twin as twin

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

MARGIN = 512
PATTERN = 0xA5
FORMATS = {"int4": 0, "int4_small": 1, "int8": 2, "mx4": 3, "mx4_h32": 4}


@pytest.fixture(scope="module")
def ops():
    from hadamard_rotated_w4a4_amd import _lib
    _lib.lib()
    return _lib


def say(msg):
    print(f"[gpu rows] {msg}", flush=True)


def guarded(nbytes):
    return torch.full((nbytes + MARGIN,), PATTERN, dtype=torch.uint8, device="cuda")


def untouched(buf, nbytes):
    return bool((buf[nbytes:] == PATTERN).all())


def rows(rng, m, k, dtype, pad=0, gain=20.0):
    """[m, k] values of a torch dtype with outlier columns, as (device view of
    rows k + pad apart, the same values as fp32 numpy)."""
    x = rng.standard_normal((m, k + pad)).astype(np.float32)
    x[:, rng.integers(0, k, max(1, k // 100))] *= gain
    t = torch.from_numpy(x).to(dtype)
    return t.cuda()[:, :k], t[:, :k].float().numpy()


def expected(fmt, v):
    if fmt.startswith("int4"):
        q, s = twin.int_rows(v, 7)
        return twin.int4_bytes(q), s
    if fmt == "int8":
        return twin.int_rows(v, 127)
    return twin.mx4_rows(v, fmt == "mx4_h32")


class Outputs:
    """Guarded code, scale and operand buffers of a format."""

    def __init__(self, ops, fmt, m, k, operand):
        self.ops, self.fmt, self.f, self.m, self.k = ops, fmt, FORMATS[fmt], m, k
        L = ops.lib()
        self.nc, self.ns = L.w4a4_act_format_code_bytes(self.f, m, k), L.w4a4_act_format_scale_bytes(self.f, m, k)
        self.no = L.w4a4_act_format_operand_bytes(self.f, m, k) if operand else 0
        self.c, self.s, self.o = guarded(self.nc), guarded(self.ns), guarded(self.no) if operand else None
        mx = fmt.startswith("mx4")
        self.args = dict(codes=self.c.view(torch.int8) if fmt == "int8" else self.c,
                         scales=self.s if mx else self.s.view(torch.float32))
        if operand:
            self.args["operand"] = self.o

    def check(self, v):
        torch.cuda.synchronize()
        codes, scales = expected(self.fmt, v)
        c, s = self.c[:self.nc].cpu().numpy(), self.s[:self.ns].cpu().numpy()
        bad = np.flatnonzero(c != np.ascontiguousarray(codes).view(np.uint8).reshape(-1))
        assert bad.size == 0, f"{bad.size} of {c.size} code bytes differ, first at {bad[:4]}"
        assert np.array_equal(s, np.ascontiguousarray(scales).view(np.uint8).reshape(-1)), "scales differ"
        assert untouched(self.c, self.nc) and untouched(self.s, self.ns)
        if self.o is not None:
            ref = torch.zeros(self.no, dtype=torch.uint8, device="cuda")
            vd = torch.from_numpy(np.ascontiguousarray(v)).cuda()
            {"int4": self.ops.rotate_quantize_prepare, "int4_small": self.ops.rotate_quantize_prepare_small,
             "int8": self.ops.rotate_quantize_prepare8}[self.fmt](vd, ref)
            torch.cuda.synchronize()
            assert torch.equal(self.o[:self.no], ref), "operand differs from the quantiser's"
            assert untouched(self.o, self.no)


# ------------------------------------------------------------------ MXFP4

@pytest.mark.parametrize("m,k,dtype,pad,rotate", [(1, 32, "f32", 0, True), (3, 96, "bf16", 0, False), (5, 256, "f16", 3, True),
                                                 (7, 288, "f32", 8, False), (33, 5120, "f16", 0, True), (130, 1056, "bf16", 8, True),
                                                 (2, 17408, "f32", 0, True)])
def test_quantize_mx4(ops, m, k, dtype, pad, rotate):
    say(f"quantize_mx4 m={m} k={k} {dtype} pad={pad} rotate={rotate}")
    x, xn = rows(np.random.default_rng(m + k), m, k, twin.TORCH[dtype], pad)
    out = Outputs(ops, "mx4_h32" if rotate else "mx4", m, k, False)
    ops.quantize_mx4(x, rotate=rotate, **out.args)
    out.check(xn)


def test_mx4_every_rounding_border_and_scale(ops):
    """Each E2M1 border, its fp32 neighbours and both signs, under every scale
    that fp32 inputs can give, subnormal blocks included."""
    borders = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7.5], np.float32)
    exps = np.arange(-149, 126)
    v = np.zeros((exps.size * 3, 32), np.float32)
    with np.errstate(over="ignore", under="ignore"):
        for i, e in enumerate(exps):
            for j, to in enumerate((0.0, np.inf, -np.inf)):
                b = borders if j == 0 else np.nextafter(borders, np.float32(to))
                row = np.concatenate((b, -b)).astype(np.float64)
                row[12] = 4.0  # fixes the scale at 2^e
                v[3 * i + j] = np.ldexp(row, e).astype(np.float32)
    say(f"quantize_mx4 borders, {v.shape[0]} blocks")
    out = Outputs(ops, "mx4", v.shape[0], 32, False)
    ops.quantize_mx4(torch.from_numpy(v).cuda(), rotate=False, **out.args)
    out.check(v)


def test_mx4_blocks_without_finite_values(ops):
    v = np.random.default_rng(0).standard_normal((4, 96)).astype(np.float32)
    v[0, 40], v[1, 33], v[2, 64:] = np.nan, np.inf, -np.inf
    say("quantize_mx4 with NaN and infinities")
    for rotate in (False, True):
        out = Outputs(ops, "mx4_h32" if rotate else "mx4", 4, 96, False)
        ops.quantize_mx4(torch.from_numpy(v).cuda(), rotate=rotate, **out.args)
        out.check(v)
        back = ops.dequantize_act(out.c[:out.nc].reshape(4, 48), out.s[:out.ns].reshape(4, 8), 96, ops.ACT_MX4).cpu().numpy()
        nan = np.isnan(back).reshape(4, 3, 32)
        assert (nan.all(-1) == nan.any(-1)).all() and nan.all(-1).tolist() == [[False, True, False], [False, True, False],
                                                                             [False, False, True], [False] * 3]


# -------------------------------------------------------------- read-back

@pytest.mark.parametrize("fmt", ["int4", "int8", "mx4"])
@pytest.mark.parametrize("m,k,dtype,pad", [(1, 32, "f32", 0), (5, 160, "f16", 0), (17, 288, "bf16", 5), (40, 5120, "f16", 8)])
def test_dequantize_act(ops, fmt, m, k, dtype, pad):
    say(f"dequantize_act {fmt} m={m} k={k} {dtype} pad={pad}")
    v = np.random.default_rng(k).standard_normal((m, k)).astype(np.float32) * 3
    codes, scales = expected(fmt, v)
    want = twin.rounded(twin.read_back(fmt, codes, scales, k), twin.TORCH[dtype])
    y = torch.full((m + 1, k + pad), 7.0, dtype=twin.TORCH[dtype], device="cuda")
    ops.dequantize_act(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), k, FORMATS[fmt], out=y[:m, :k])
    torch.cuda.synchronize()
    got = y.float().cpu().numpy()
    assert np.array_equal(got[:m, :k], want)
    assert (got[m:] == 7).all() and (got[:, k:] == 7).all()


def test_read_back_of_every_scale_byte(ops):
    codes = np.tile(np.arange(16, dtype=np.uint8) | np.arange(16, dtype=np.uint8)[::-1] << 4, (256, 1))
    scales = np.full((256, 8), 127, np.uint8)
    scales[:, 0] = np.arange(256)
    y = ops.dequantize_act(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 32, ops.ACT_MX4).cpu().numpy()
    with np.errstate(over="ignore"):
        want = twin.mx4_values(codes, scales, 32).astype(np.float32)
    assert np.array_equal(y, want, equal_nan=True)


# ------------------------------------------------------------------- norm

NORM_SIZES = [(1, 32), (1, 5120), (3, 96), (16, 160), (33, 2048), (2, 8224), (2, 16416), (2, 32800), (70, 768)]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("m,k", NORM_SIZES)
def test_norm_formats_and_sizes(ops, fmt, m, k):
    if fmt == "int4_small":
        m = min(m, 16)
    say(f"rms_norm_quantize {fmt} m={m} k={k}")
    rng = np.random.default_rng(m * 7 + k)
    x, xn = rows(rng, m, k, torch.float32)
    r, rn = rows(rng, m, k, torch.float16)
    w = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    hn, v = twin.norm(xn, rn, torch.float16, w, 1e-6)
    for operand in ([True] if fmt == "int4_small" else [False] if fmt.startswith("mx4") else [False, True]):
        out = Outputs(ops, fmt, m, k, operand)
        _, _, h = ops.rms_norm_quantize(x, torch.from_numpy(w).cuda(), 1e-6, FORMATS[fmt], residual=r, **out.args)
        out.check(v)
        assert np.array_equal(h.float().cpu().numpy(), hn)


@pytest.mark.parametrize("xdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rdt", ["f32", "f16", "bf16"])
def test_norm_types_and_strides(ops, xdt, rdt):
    say(f"rms_norm_quantize x {xdt}, residual {rdt}")
    rng = np.random.default_rng(5)
    for m, k, px, pr, ph in ((9, 352, 0, 0, 0), (9, 352, 1, 3, 5), (20, 1024, 8, 16, 8)):
        x, xn = rows(rng, m, k, twin.TORCH[xdt], px)
        r, rn = rows(rng, m, k, twin.TORCH[rdt], pr)
        wbuf = torch.from_numpy((1 + 0.1 * rng.standard_normal(k + 1)).astype(np.float32)).cuda()
        w = wbuf[1:] if px == 1 else wbuf[:k]  # 4-byte and 16-byte aligned weights
        hn, v = twin.norm(xn, rn, twin.TORCH[rdt], w.cpu().numpy(), 1e-5)
        hbuf = torch.full((m + 1, k + ph), 7.0, dtype=twin.TORCH[rdt], device="cuda")
        out = Outputs(ops, "mx4_h32", m, k, False)
        ops.rms_norm_quantize(x, w, 1e-5, ops.ACT_MX4_H32, residual=r, h=hbuf[:m, :k], **out.args)
        out.check(v)
        got = hbuf.float().cpu().numpy()
        assert np.array_equal(got[:m, :k], hn) and (got[m:] == 7).all() and (got[:, k:] == 7).all()


@pytest.mark.parametrize("k", [2048, 33024])  # held in registers, and walked twice
def test_norm_in_place_and_without_residual_or_weight(ops, k):
    rng = np.random.default_rng(11)
    m = 6
    say(f"rms_norm_quantize in place, k={k}")
    w = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    x, xn = rows(rng, m, k, torch.bfloat16)
    r, rn = rows(rng, m, k, torch.bfloat16)
    hn, v = twin.norm(xn, rn, torch.bfloat16, w, 1e-6)
    for target in ("residual", "x"):
        xc, rc = x.clone(), r.clone()
        out = Outputs(ops, "int8", m, k, False)
        ops.rms_norm_quantize(xc, torch.from_numpy(w).cuda(), 1e-6, ops.ACT_INT8, residual=rc,
                              h=rc if target == "residual" else xc, **out.args)
        out.check(v)
        assert np.array_equal((rc if target == "residual" else xc).float().cpu().numpy(), hn)
        assert torch.equal(xc if target == "residual" else rc, x if target == "residual" else r)
    # no residual, no weight: the norm of x itself, nothing written but the rows
    _, v = twin.norm(xn, None, torch.bfloat16, None, 1e-6)
    out = Outputs(ops, "int4", m, k, False)
    codes, scales, h = ops.rms_norm_quantize(x, None, 1e-6, ops.ACT_INT4, **out.args)
    out.check(v)
    assert h is None
    # no residual, h of another type: the norm reads what h holds
    xf, xfn = rows(rng, m, k, torch.float32)
    hn, v = twin.norm(xfn, None, torch.float16, w, 1e-6)
    hb = torch.empty((m, k), dtype=torch.float16, device="cuda")
    out = Outputs(ops, "mx4", m, k, False)
    ops.rms_norm_quantize(xf, torch.from_numpy(w).cuda(), 1e-6, ops.ACT_MX4, h=hb, **out.args)
    out.check(v)
    assert np.array_equal(hb.float().cpu().numpy(), hn)


def test_norm_of_zero_tiny_and_huge_rows(ops):
    """Zero rows (eps keeps the root finite), rows whose squares pass fp32's
    range on both ends, and rows that cancel to zero with their residual."""
    m, k = 6, 512
    x = np.random.default_rng(3).standard_normal((m, k)).astype(np.float32)
    r = np.zeros_like(x)
    x[0] = 0
    x[1] *= np.float32(1e30)
    x[2] *= np.float32(1e-30)
    r[3] = -x[3]
    x[4] *= np.float32(3e37)
    say("rms_norm_quantize extreme rows")
    for fmt in ("int8", "mx4_h32"):
        hn, v = twin.norm(x, r, torch.float32, None, 1e-6)
        out = Outputs(ops, fmt, m, k, False)
        _, _, h = ops.rms_norm_quantize(torch.from_numpy(x).cuda(), None, 1e-6, FORMATS[fmt], residual=torch.from_numpy(r).cuda(),
                                        **out.args)
        out.check(v)
        assert np.array_equal(h.cpu().numpy(), hn)


# ------------------------------------------------------- gated activation

@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,k,dtype,pad", [(1, 32, "f32", 0), (16, 1056, "f32", 0), (13, 96, "bf16", 1), (45, 768, "f16", 768)])
def test_glu(ops, fmt, act, m, k, dtype, pad):
    if fmt == "int4_small":
        m = min(m, 16)
    say(f"glu_quantize {fmt} {act} m={m} k={k} {dtype} pad={pad}")
    rng = np.random.default_rng(m + k)
    g, gn = rows(rng, m, k, twin.TORCH[dtype], pad)
    u, un = rows(rng, m, k, twin.TORCH[dtype], 0, 1.0)
    if pad == k:  # one packed gate|up matrix
        both = torch.cat((g, u), 1)
        g, u = both[:, :k], both[:, k:]
    v = twin.gated(gn, un, getattr(twin, act))
    for operand in ([True] if fmt == "int4_small" else [False] if fmt.startswith("mx4") else [False, True]):
        out = Outputs(ops, fmt, m, k, operand)
        ops.glu_quantize(g, u, FORMATS[fmt], act=ops.GLU_SILU if act == "silu" else ops.GLU_GELU_TANH, **out.args)
        out.check(v)


def test_glu_over_the_range_of_the_gate(ops):
    """Gates from -1e4 to 1e4 and near zero: where e^-g under- and overflows
    fp32, and where the result is a subnormal."""
    g = np.concatenate((np.linspace(-120, 120, 4064), [-1e4, 1e4, -0.0, 0.0, 1e-40, -1e-40, 88.8, -88.8, 103.9, -103.9, -87.3, 745.0,
                                                       -745.0, 710.0, -710.0, 1e-20, -1e-20, 30.0, -30.0, 17.0, -17.0, 6.0, -6.0,
                                                       3.0, -3.0, 1.0, -1.0, 0.5, -0.5, 5e-3, -5e-3, 2.0])).astype(np.float32)
    g = g.reshape(-1, 32)[:, np.random.default_rng(0).permutation(32)].copy()
    u = np.random.default_rng(1).standard_normal(g.shape).astype(np.float32)
    for act in ("silu", "gelu_tanh"):
        say(f"glu_quantize gate range {act}")
        v = twin.gated(g, u, getattr(twin, act))
        out = Outputs(ops, "int8", g.shape[0], 32, False)
        ops.glu_quantize(torch.from_numpy(g).cuda(), torch.from_numpy(u).cuda(), ops.ACT_INT8,
                         act=ops.GLU_SILU if act == "silu" else ops.GLU_GELU_TANH, **out.args)
        out.check(v)


# ----------------------------------------------------------------- empties

def test_empty_rows(ops):
    x = torch.zeros((0, 64), device="cuda")
    assert ops.quantize_mx4(x)[0].shape == (0, 32)
    assert ops.rms_norm_quantize(x, None, 1e-6, ops.ACT_MX4, residual=x)[2].shape == (0, 64)
    assert ops.glu_quantize(x, x, ops.ACT_INT8)[0].shape == (0, 64)
    z = torch.zeros((4, 0), device="cuda")
    assert ops.quantize_mx4(z)[1].shape == (4, 0)
    assert ops.dequantize_act(torch.zeros((4, 0), dtype=torch.uint8, device="cuda"), torch.zeros((4, 0), dtype=torch.uint8, device="cuda"), 0, ops.ACT_MX4).shape == (4, 0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("m,k", [(512, 4128), (515, 5120), (600, 8224), (511, 4128), (1030, 96)])
def test_norm_of_many_rows(ops, m, k):
    """From 512 rows a thread holds more of a row."""
    say(f"rms_norm_quantize m={m} k={k}")
    rng = np.random.default_rng(m + k)
    x, xn = rows(rng, m, k, torch.float32)
    r, rn = rows(rng, m, k, torch.bfloat16)
    w = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    hn, v = twin.norm(xn, rn, torch.bfloat16, w, 1e-6)
    for fmt, operand in (("int8", False), ("int4", True)):
        out = Outputs(ops, fmt, m, k, operand)
        _, _, h = ops.rms_norm_quantize(x, torch.from_numpy(w).cuda(), 1e-6, FORMATS[fmt], residual=r, **out.args)
        out.check(v)
        assert np.array_equal(h.float().cpu().numpy(), hn)


def test_rows_past_32_bit_offsets(ops):
    """Tensors of more than 4 GB: the last rows and those around byte 2^32 are
    what the same rows give in a call of their own."""
    m, k = 65000, 17408
    say(f"4 GB tensors m={m} k={k}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((m, k), device="cuda")
    x.normal_(generator=g)
    edge = 2 ** 32 // (4 * k)
    spots = [slice(0, 5), slice(edge - 5, edge + 5), slice(m - 7, m)]
    w = torch.rand(k, device="cuda", generator=g)

    c, s = ops.quantize_mx4(x)
    back = ops.dequantize_act(c, s, k, ops.ACT_MX4_H32)
    for at in spots:
        c1, s1 = ops.quantize_mx4(x[at].clone())
        assert torch.equal(c[at], c1) and torch.equal(s[at], s1), at
        assert torch.equal(back[at], ops.dequantize_act(c1, s1, k, ops.ACT_MX4_H32)), at
    del back
    c, s, h = ops.rms_norm_quantize(x, w, 1e-6, ops.ACT_INT8, residual=x)
    for at in spots:
        one = x[at].clone()
        c1, s1, h1 = ops.rms_norm_quantize(one, w, 1e-6, ops.ACT_INT8, residual=one)
        assert torch.equal(c[at], c1) and torch.equal(s[at], s1) and torch.equal(h[at], h1), at
    del h
    z = x.view(torch.bfloat16)  # 2 k wide: gate and up of a joint product
    c, s = ops.glu_quantize(z[:, :k], z[:, k:], ops.ACT_MX4)
    for at in spots:
        one = z[at].clone()
        c1, s1 = ops.glu_quantize(one[:, :k], one[:, k:], ops.ACT_MX4)
        assert torch.equal(c[at], c1) and torch.equal(s[at], s1), at
    torch.cuda.synchronize()

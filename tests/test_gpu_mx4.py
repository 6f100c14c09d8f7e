"""GPU tests of the MXFP4 product, and of the new operators in a chain.

Operand values are small multiples of a common power of two, so that every
partial sum, in any order, is a whole number of units below 2^24: the fp32
result is exact and is compared for equality with the 64-bit product (rounded
once where y has 16 bits).  Wide exponent ranges are compared within the bound
of K fp32 additions, K 2^-23 sum |a w| (a whole last place each: the matrix
instruction's own rounding within its 64 products is not assumed to be to
nearest)."""
import numpy as np
import pytest

import rows_twin as twin

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from hadamard_rotated_w4a4_amd import _lib
    _lib.lib()
    return _lib


def say(msg):
    print(f"[gpu mx4] {msg}", flush=True)


def operand(rng, rows, k, lo, hi):
    """Random MXFP4 rows, scales 2^lo .. 2^hi; the padding scale bytes hold
    255 (which a reader must ignore)."""
    codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    scales = np.full((rows, twin.stride(k)), 255, np.uint8)
    scales[:, :k // 32] = rng.integers(127 + lo, 128 + hi, (rows, k // 32))
    return codes, scales


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def product(ops, rng, m, n, k, lo=-1, hi=1):
    ac, asc = operand(rng, m, k, lo, hi)
    wc, wsc = operand(rng, n, k, lo, hi)
    packed = ops.repack_mx4(dev(wc), dev(wsc), n, k)
    a = torch.from_numpy(twin.mx4_values(ac, asc, k)).cuda()
    w = torch.from_numpy(twin.mx4_values(wc, wsc, k)).cuda()
    return packed, dev(ac), dev(asc), a, w


SIZES = [(1, 1, 32), (1, 33, 96), (2, 1024, 5120), (5, 70, 288), (16, 96, 256), (16, 1024, 5120), (13, 544, 17408), (17, 100, 512),
         (32, 4096, 2048), (33, 257, 1056), (64, 5120, 1024), (100, 1000, 2080), (128, 128, 128), (129, 385, 768), (200, 2176, 5120),
         (302, 640, 17408), (512, 1536, 2048), (700, 130, 64)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_is_exact_on_small_units(ops, m, n, k):
    say(f"gemm_mx4 m={m} n={n} k={k}")
    rng = np.random.default_rng(m * 31 + n * 7 + k)
    packed, ac, asc, a, w = product(ops, rng, m, n, k)
    # units of 2^-2 2^-2: the largest sum of magnitudes is K * (6 * 2)^2 * 16 < 2^24 for K <= 7281; above, the random signs
    # keep every partial sum far below it
    want = a @ w.t().contiguous()
    bound = (a.abs() @ w.abs().t().contiguous()).max().item() * 16
    assert k > 7281 or bound < 2 ** 24
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        y = torch.full((m + 2, n + 3), 7.0, dtype=dtype, device="cuda")
        ops.gemm_mx4(packed, ac, asc, n, k, y=y[:m, :n])
        torch.cuda.synchronize()
        bad = (y[:m, :n] != want.float().to(dtype)).nonzero()
        assert bad.numel() == 0, f"{dtype}: {bad.shape[0]} of {m * n} outputs differ, first at {bad[0].tolist()}"
        assert (y[m:] == 7).all() and (y[:, n:] == 7).all()
    assert torch.equal(ops.gemm_mx4(packed, ac, asc, n, k), want.float())


@pytest.mark.parametrize("m,n,k", [(3, 64, 512), (40, 96, 1024), (256, 256, 4096)])
def test_product_over_wide_scales(ops, m, n, k):
    say(f"gemm_mx4 wide scales m={m} n={n} k={k}")
    packed, ac, asc, a, w = product(ops, np.random.default_rng(k), m, n, k, -20, 20)
    y = ops.gemm_mx4(packed, ac, asc, n, k).double()
    err = (y - a @ w.t().contiguous()).abs()
    bound = k * 2.0 ** -23 * (a.abs() @ w.abs().t().contiguous())
    assert (err <= bound).all(), f"worst {(err / bound).max().item():.3g} of the bound"


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_nan_blocks_reach_their_rows_and_columns_only(ops, m):
    n, k = 160, 544
    say(f"gemm_mx4 NaN blocks m={m}")
    rng = np.random.default_rng(m)
    ac, asc = operand(rng, m, k, -1, 1)
    wc, wsc = operand(rng, n, k, -1, 1)
    asc[m // 2, 3], wsc[35, 16] = 255, 255
    y = ops.gemm_mx4(ops.repack_mx4(dev(wc), dev(wsc), n, k), dev(ac), dev(asc), n, k).cpu().numpy()
    nan = np.isnan(y)
    want = np.zeros((m, n), bool)
    want[m // 2], want[:, 35] = True, True
    assert np.array_equal(nan, want)
    ref = np.nan_to_num(twin.mx4_values(ac, asc, k)) @ np.nan_to_num(twin.mx4_values(wc, wsc, k)).T
    assert np.array_equal(y[~want], ref[~want].astype(np.float32))


def test_extreme_scales(ops):
    """Scales at both ends: products below fp32's range vanish or round into
    the subnormals, sums past it are infinite."""
    k, n = 64, 32
    ac = np.full((3, k // 2), 0x22, np.uint8)  # every element 1.0
    wc = np.full((n, k // 2), 0x22, np.uint8)
    asc, wsc = np.full((3, 8), 127, np.uint8), np.full((n, 8), 127, np.uint8)
    asc[0, :2], asc[1, :2] = 0, 254
    wsc[1, :2], wsc[2, :2] = 254, 0
    y = ops.gemm_mx4(ops.repack_mx4(dev(wc), dev(wsc), n, k), dev(ac), dev(asc), n, k).cpu().numpy()
    assert y[2, 0] == 64 and y[2, 1] == np.inf and y[2, 2] == np.float32(64 * 2.0 ** -127)
    assert y[0, 0] == np.float32(64 * 2.0 ** -127) and y[0, 1] == 64 and y[0, 2] == 0
    assert y[1, 0] == np.inf and y[1, 1] == np.inf and y[1, 2] == 64


def test_empty_product(ops):
    z = torch.empty(0, dtype=torch.uint8, device="cuda")
    y = torch.full((4, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((4, 0), dtype=torch.uint8, device="cuda")
    ops.gemm_mx4(z, e, e, 6, 0, y=y[:, :6])
    assert (y[:, :6] == 0).all() and (y[:, 6:] == 7).all()
    assert ops.gemm_mx4(z, torch.empty((0, 32), dtype=torch.uint8, device="cuda"), torch.empty((0, 8), dtype=torch.uint8, device="cuda"), 5, 64).shape == (0, 5)


# ------------------------------------------------------------ in a chain

def weights(rng, n, k):
    return (rng.standard_normal((n, k)) * 0.02).astype(np.float32)


class Layer:
    """norm -> gate|up -> gated activation -> down -> norm with the residual,
    every stage on MXFP4 rows."""

    def __init__(self, ops, d, ff, rng):
        self.ops, self.d, self.ff = ops, d, ff
        self.w_gu, self.w_dn = (dev(weights(rng, n, k)) for n, k in ((2 * ff, d), (d, ff)))
        self.gu, self.dn = ops.prepare_weights_mx4(self.w_gu), ops.prepare_weights_mx4(self.w_dn)
        self.g1, self.g2 = (dev((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)) for _ in range(2))

    def __call__(self, x, residual):
        ops, d, ff = self.ops, self.d, self.ff
        c1, s1, h1 = ops.rms_norm_quantize(x, self.g1, 1e-6, ops.ACT_MX4_H32, residual=residual)
        z = ops.gemm_mx4(self.gu, c1, s1, 2 * ff, d, dtype=torch.bfloat16)
        c2, s2 = ops.glu_quantize(z[:, :ff], z[:, ff:], ops.ACT_MX4_H32)
        o = ops.gemm_mx4(self.dn, c2, s2, d, ff)
        c3, s3, h2 = ops.rms_norm_quantize(o, self.g2, 1e-6, ops.ACT_INT8, residual=h1)
        return dict(c1=c1, s1=s1, h1=h1, z=z, c2=c2, s2=s2, o=o, c3=c3, s3=s3, h2=h2)


def layer_inputs(m, d, seed):
    rng = np.random.default_rng(seed)
    return dev(rng.standard_normal((m, d)).astype(np.float32)), dev(rng.standard_normal((m, d)).astype(np.float32)).bfloat16()


@pytest.mark.parametrize("m,d,ff", [(1, 1024, 2816), (16, 512, 768), (45, 512, 1376), (300, 1024, 768)])
def test_a_feed_forward_layer(ops, m, d, ff):
    """Each stage against the plain form of that stage on what reached it."""
    say(f"layer m={m} d={d} ff={ff}")
    layer = Layer(ops, d, ff, np.random.default_rng(m))
    x, r = layer_inputs(m, d, 1)
    t = layer(x, r)
    torch.cuda.synchronize()
    n = {name: v.float().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for name, v in t.items()}
    h, v = twin.norm(x.cpu().numpy(), r.float().cpu().numpy(), torch.bfloat16, layer.g1.cpu().numpy(), 1e-6)
    assert np.array_equal(n["h1"], h)
    c, s = twin.mx4_rows(v, True)
    assert np.array_equal(n["c1"], c) and np.array_equal(n["s1"], s)

    def held(got, codes, scales, w, k, half_step):
        a = torch.from_numpy(twin.mx4_values(codes, scales, k))
        b = torch.from_numpy(twin.mx4_values(*twin.mx4_rows(w.cpu().numpy(), True), k))
        want, size = a @ b.t(), a.abs() @ b.abs().t()
        bound = (k * 2.0 ** -23 * size) * (1 + half_step) + half_step * want.abs()
        assert ((torch.from_numpy(got).double() - want).abs() <= bound).all()

    held(n["z"], c, s, layer.w_gu, d, 2.0 ** -8)
    v = twin.gated(n["z"][:, :ff], n["z"][:, ff:], twin.silu)
    c, s = twin.mx4_rows(v, True)
    assert np.array_equal(n["c2"], c) and np.array_equal(n["s2"], s)
    held(n["o"], c, s, layer.w_dn, ff, 0.0)
    h, v = twin.norm(n["o"], n["h1"], torch.bfloat16, layer.g2.cpu().numpy(), 1e-6)
    q, s = twin.int_rows(v, 127)
    assert np.array_equal(n["h2"], h) and np.array_equal(n["c3"], q) and np.array_equal(n["s3"], s)


@pytest.mark.parametrize("m", [1, 16, 200])
def test_the_layer_captured_and_replayed(ops, m):
    say(f"layer graph m={m}")
    d, ff = 1024, 1376
    layer = Layer(ops, d, ff, np.random.default_rng(3))
    x, r = layer_inputs(m, d, 0)
    eager, inputs = [], [layer_inputs(m, d, seed) for seed in (5, 6, 7)]
    for xi, ri in inputs:
        x.copy_(xi)
        r.copy_(ri)
        eager.append({name: v.clone() for name, v in layer(x, r).items()})
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = layer(x, r)
    torch.cuda.synchronize()
    for rep in range(2):
        for (xi, ri), want in zip(inputs, eager):
            x.copy_(xi)
            r.copy_(ri)
            other = layer(xi, ri)  # eager work between the replays
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for name, v in out.items():
                assert torch.equal(v, want[name]), f"replay {rep}: {name}"
                assert torch.equal(other[name], want[name])


def test_two_streams_at_once(ops):
    say("layers on two streams")
    d, ff = 512, 768
    layer = Layer(ops, d, ff, np.random.default_rng(4))
    inputs = [layer_inputs(m, d, m) for m in (16, 300)]
    want = [layer(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = [[], []]
    for _ in range(4):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[j].append(layer(*inputs[j]))
    torch.cuda.synchronize()
    for j in range(2):
        for t in got[j]:
            for name, v in t.items():
                assert torch.equal(v, want[j][name]), (j, name)


def test_results_do_not_depend_on_the_other_rows(ops):
    """A row's outputs are the same alone, among 16 and among 300 rows, for
    operands whose sums are exact."""
    n, k = 544, 1024
    packed, ac, asc, _, _ = product(ops, np.random.default_rng(9), 300, n, k)
    whole = ops.gemm_mx4(packed, ac, asc, n, k)
    for m in (1, 16, 33):
        assert torch.equal(ops.gemm_mx4(packed, ac[:m], asc[:m], n, k), whole[:m])


def device_operand(g, rows, k):
    """Random rows with scales of 2^-1 and 1, and their values in 64 bits; the
    padding scale bytes hold 255."""
    codes = torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((rows, twin.stride(k)), 255, dtype=torch.uint8, device="cuda")
    scales[:, :k // 32] = torch.randint(126, 128, (rows, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales


def values(ops, codes, scales, k):
    return ops.dequantize_act(codes, scales, k, ops.ACT_MX4).double()


# every tile shape, whole, with K splits and with the rest in a second shape;
# streams of 16, 32 and 64 rows, short and long K, one and several row blocks
PLANS = [(65, 5101, 17408), (130, 5101, 8224), (302, 10201, 96), (65, 34801, 96), (65, 10201, 17408),
         (302, 34801, 5152), (200, 34801, 96), (400, 10201, 17408), (700, 17401, 96), (200, 17401, 17408),
         (400, 34801, 1056), (700, 34801, 2080), (302, 5101, 17408), (300, 10208, 8224), (33, 17401, 17408),
         (65, 8225, 17408), (450, 2081, 17408), (150, 34801, 5152), (1000, 5101, 17408), (400, 17401, 96),
         (1000, 20513, 5152), (16, 9001, 5120), (9, 9001, 17408), (20, 9001, 5120), (27, 1000, 17408),
         (50, 8161, 5152), (250, 2041, 5152), (1000, 481, 2080), (4090, 130, 544)]


@pytest.mark.parametrize("m,n,k", PLANS)
def test_product_of_every_plan(ops, m, n, k):
    """Exact, as above: units of 2^-4, sums of 17408 random products of at
    most 36 whole units of 1 stay far below 2^20."""
    say(f"gemm_mx4 plan m={m} n={n} k={k}")
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    (ac, asc), (wc, wsc) = device_operand(g, m, k), device_operand(g, n, k)
    packed = ops.repack_mx4(wc, wsc, n, k)
    want = (values(ops, ac, asc, k) @ values(ops, wc, wsc, k).t().contiguous()).float()
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((m + 1, n + 7), 7.0, dtype=dtype, device="cuda")
        ops.gemm_mx4(packed, ac, asc, n, k, y=y[:m, :n])
        torch.cuda.synchronize()
        bad = (y[:m, :n] != want.to(dtype)).nonzero()
        assert bad.numel() == 0, f"{dtype}: {bad.shape[0]} of {m * n} outputs differ, first at {bad[0].tolist()}"
        assert (y[m:] == 7).all() and (y[:, n:] == 7).all()


def test_outputs_past_32_bit_offsets(ops):
    m, n, k = 33000, 34816, 96
    say(f"gemm_mx4 4 GB outputs m={m} n={n} k={k}")
    g = torch.Generator(device="cuda").manual_seed(3)
    (ac, asc), (wc, wsc) = device_operand(g, m, k), device_operand(g, n, k)
    packed = ops.repack_mx4(wc, wsc, n, k)
    y = ops.gemm_mx4(packed, ac, asc, n, k)
    for at in (slice(0, 40), slice(2 ** 32 // (4 * n) - 20, 2 ** 32 // (4 * n) + 20), slice(m - 40, m)):
        assert torch.equal(y[at], ops.gemm_mx4(packed, ac[at].clone(), asc[at].clone(), n, k)), at


def test_weights_past_32_bit_offsets(ops):
    n, k = 500000, 17408
    say(f"repack_mx4 and gemm_mx4 4 GB weights n={n} k={k}")
    g = torch.Generator(device="cuda").manual_seed(4)
    wc, wsc = device_operand(g, n, k)
    packed = ops.repack_mx4(wc, wsc, n, k)
    assert packed.numel() > 2 ** 32
    edge = 2 ** 32 // (k // 2)  # the plain codes' row there
    last = 2 ** 32 // (packed.numel() // ((n + 31) // 32)) * 32  # the records' first row there
    for m in (1, 30, 70):
        ac, asc = device_operand(g, m, k)
        y = ops.gemm_mx4(packed, ac, asc, n, k)
        a = values(ops, ac, asc, k)
        for at in (slice(0, 40), slice(edge - 20, edge + 20), slice(last - 20, last + 20), slice(n - 40, n)):
            want = a @ values(ops, wc[at].clone(), wsc[at].clone(), k).t().contiguous()
            assert torch.equal(y[:, at], want.float()), (m, at)

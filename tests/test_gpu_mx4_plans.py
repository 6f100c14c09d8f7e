"""Every plan of the MXFP4 product is run by a test: the sizes below, with those of
test_gpu_mx4, reach each kernel shape whole, with K splits, ahead of another
shape and as the remaining columns of one.  The CPU test holds the list against
the plans that a sweep of sizes gives, so a refit of the plan's constants shows
here which sizes have to join."""
import ctypes
import math
import random
import re

import pytest

from test_gpu_mx4 import PLANS, SIZES, device_operand, values

torch = pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import _lib as ops  # noqa: E402

MORE = [(208, 21908, 32), (384, 17408, 5120), (385, 17411, 1056), (196, 24441, 32),  # 128x128
        (67, 24807, 15520), (77, 12791, 19232),  # 128x128, splits
        (378, 25793, 2272), (365, 25902, 2720), (258, 33168, 10304), (180, 37347, 5344),  # rests of the smaller shapes
        (614, 29093, 2368), (771, 18479, 14784), (805, 17123, 10848), (3455, 7044, 1600),  # 256x192 and a rest
        (3368, 11120, 960), (1876, 18478, 704), (692, 22347, 832), (2632, 13337, 800), (1999, 13855, 1664),  # 256x256 and a rest
        (152, 10280, 18048), (129, 8727, 13792), (129, 5585, 13952),  # 160x128, splits
        (74, 4358, 6720), (35, 9524, 6304), (33, 8546, 6048), (65, 4109, 10560), (68, 8621, 8512),  # 64x64, splits
        (242, 17983, 19680), (453, 8032, 19552), (225, 19022, 19744)]  # large tiles, splits


def kind(size):
    """A plan without the number of its splits."""
    return re.sub(r"split \d+", "split", ops.gemm_mx4_plan(*size))


def sweep(count):
    rng = random.Random(1)

    def spread(lo, hi):
        return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    return [(spread(1, 4096), spread(1, 40000), 32 * spread(1, 640)) for _ in range(count)]


def test_every_plan_of_a_sweep_is_run_by_a_test():
    tested = {kind(s) for s in PLANS + SIZES + MORE}
    missing = {}
    for s in sweep(60000):
        if kind(s) not in tested:
            missing.setdefault(kind(s), s)
    assert not missing, f"plans that no GPU test runs, each with a size: {missing}"


def test_every_shape_is_run_in_each_of_its_places():
    texts = [ops.gemm_mx4_plan(*s) for s in PLANS + SIZES + MORE]
    shapes = {"64x64", "64x128", "128x128", "160x128", "256x192", "256x256"}
    assert {t for t in texts if t.startswith("stream")} == {"stream 16x8", "stream 16x16", "stream 32x8", "stream 32x16", "stream 64x16"}
    assert {t.split()[1] for t in texts if t.startswith("tile") and len(t.split()) == 2} == shapes
    assert {t.split()[1] for t in texts if "+" in t} == shapes - {"64x64"}
    assert {t.split()[3] for t in texts if "+" in t} == shapes - {"256x256"}
    assert {t.split()[1] for t in texts if "split" in t} >= {"64x64", "128x128", "160x128", "256x192", "256x256"}


def test_plan_query():
    """As the workspace: nothing for empty or invalid sizes, cut off like snprintf."""
    L = ops.lib()
    for bad in ((0, 64, 64), (64, 0, 64), (64, 64, 0), (64, 64, 48), (-1, 64, 64), (65535 * 32 + 1, 64, 64), (1, 1, 1 << 25)):
        assert ops.gemm_mx4_plan(*bad) == ""
    for m, n, k in PLANS + SIZES + MORE:
        text, need = ops.gemm_mx4_plan(m, n, k), ops.gemm_mx4_workspace_bytes(m, n, k)
        assert text.startswith("stream") == (need == 0)
        rows = (ops.mx4_packed_bytes(m, k) + 255) // 256 * 256 if need else 0
        splits = int(text.split()[-1]) if "split" in text else 0
        assert need == rows + (splits * m * n * 4 + 255) // 256 * 256
    assert L.w4a4_gemm_mx4_plan(1, 1, 32, None, 0) == len("stream 16x8") == L.w4a4_gemm_mx4_plan(1, 1, 32, None, 9)
    short = ctypes.create_string_buffer(7)
    assert L.w4a4_gemm_mx4_plan(1, 1, 32, short, 7) == len("stream 16x8") and short.value == b"stream"


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", MORE)
def test_product_of_each_further_plan(m, n, k):
    """Exact: units of 2^-4, sums of at most 19744 random products of at most 36
    whole units of 1 stay far below 2^20."""
    print(f"[gpu mx4] {ops.gemm_mx4_plan(m, n, k)}: m={m} n={n} k={k}", flush=True)
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

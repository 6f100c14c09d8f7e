"""The paged 8-bit key/value cache and attention over it, on the GPU, against
the definitions written a second time in numpy (kv_twin)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_twin as twin  # noqa: E402
from hadamard_rotated_w4a4_amd import ops  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def page_table(rng, per_seq, pool, width=None):
    """Every sequence's pages, drawn from the pool without repeats; -1 behind them."""
    order, at, width = rng.permutation(pool), 0, width or max(per_seq + [1])
    out = np.full((len(per_seq), width), -1, np.int32)
    for b, n in enumerate(per_seq):
        out[b, :n] = order[at:at + n]
        at += n
    return out


def filled(rng, pool, page, heads, dim):
    """A pool of finite codes (no NaN) and scales near 1."""
    codes = rng.integers(0, 256, (pool, heads, page // 32, 2, 32 * dim)).astype(np.uint8)
    codes[codes & 127 == 127] -= 1
    return codes, rng.integers(117, 123, (pool, heads, page // 32, 2)).astype(np.uint8)


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def rope_table(n, width):
    half = width // 2
    angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32)


# (page, heads, q heads, dim), then (rows, tokens) of each sequence
APPENDS = [
    ((32, 1, 1, 64), [(1, 1)]),
    ((32, 2, 6, 256), [(1, 33), (1, 64), (0, 7), (1, 31)]),
    ((64, 3, 3, 128), [(5, 37), (40, 40), (65, 130), (0, 0)]),
    ((96, 2, 4, 64), [(32, 32), (97, 200), (3, 2), (2, 0)]),  # more rows than tokens
    ((128, 4, 8, 128), [(200, 333)]),
]


@pytest.mark.parametrize("shape,seqs", APPENDS)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["plain", "halves", "pairs norm", "axes norm"])
def test_append_writes_the_codes_of_the_definition(shape, seqs, dt, form):
    page, heads, q_heads, dim = shape
    rng = np.random.default_rng([page, heads, dim, len(form)])
    pool = sum(-(-t // page) for _, t in seqs) + 2
    pages = page_table(rng, [-(-t // page) for _, t in seqs], pool)
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    rows, lens = int(starts[-1]) + 2, np.array([t for _, t in seqs], np.int32)  # two rows behind the last sequence
    codes, scales = filled(rng, pool, page, heads, dim)
    x = torch.from_numpy((rng.standard_normal((rows, q_heads + 2 * heads, dim)) * np.exp(rng.standard_normal((rows, 1, 1)))).astype(np.float32))
    x[:, :, ::37] *= 30
    x = x.to(TYPES[dt])
    q, k, v = (x.float().numpy()[:, a:b] for a, b in ((0, q_heads), (q_heads, q_heads + heads), (q_heads + heads, q_heads + 2 * heads)))
    given = {}
    if form != "plain":
        width = dim if form == "halves" else 16 if form == "pairs norm" else dim // 2
        given = {"rope": rope_table(400, width), "interleaved": form == "pairs norm"}
        if form == "axes norm":
            given["positions"] = rng.integers(0, 400, (3, rows)).astype(np.int32)
            given["axes"] = (np.arange(width // 2) % 3).astype(np.uint8)
    if "norm" in form:
        given["q_weight"] = (1 + 0.1 * rng.standard_normal(dim)).astype(np.float32)
        given["k_weight"] = (1 + 0.1 * rng.standard_normal(dim)).astype(np.float32)
    c, s, xs = gpu(codes), gpu(scales), x.to(DEV)
    out = torch.full((rows, q_heads, dim), 9.0, dtype=torch.float16, device=DEV)
    on_gpu = {n: y if isinstance(y, bool) else gpu(y) for n, y in given.items()}
    got = ops.append_kv(xs[:, q_heads:q_heads + heads], xs[:, q_heads + heads:], c, s, gpu(pages), ints(starts.tolist()), gpu(lens),
                        q=xs[:, :q_heads], q_out=out, **on_gpu)
    assert got is out
    want = twin.append(k, v, codes, scales, pages, starts, lens, q=q, **given)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(c.cpu().numpy(), codes)
    expected = torch.from_numpy(want).to(torch.float16)
    expected[-2:] = 9.0
    same = (out.cpu() == expected) | (torch.isnan(out.cpu()) & torch.isnan(expected))
    assert bool(same.all())


def test_read_gives_what_the_codes_stand_for():
    rng = np.random.default_rng(5)
    for dim, page, seqs in ((64, 64, [(3, 70), (0, 5), (33, 33)]), (128, 32, [(1, 1), (50, 96), (4, 2)]), (256, 96, [(130, 200)])):
        per = [-(-t // page) for _, t in seqs]
        pool = sum(per) + 1
        codes, scales = filled(rng, pool, page, 2, dim)
        pages = page_table(rng, per, pool)
        if dim == 128:
            pages[1, 1] = 77  # no page: its tokens read as zeros
        starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
        rows, lens = int(starts[-1]), np.array([t for _, t in seqs], np.int32)
        want = twin.read(codes, scales, pages, starts, lens, rows)
        args = gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens)
        for dt in (torch.float32, torch.bfloat16, torch.float16):
            k, v = ops.read_kv(*args, rows, dtype=dt)
            for got, exact in ((k, want[0]), (v, want[1])):
                assert torch.equal(got.cpu(), torch.from_numpy(exact.astype(np.float32)).to(dt))
        wide = torch.full((2, rows + 1, 3, dim), 5.0, device=DEV)  # outputs with room between heads and behind the rows
        ops.read_kv(*args, rows, k=wide[0][:rows, :2], v=wide[1][:rows, 1:])
        assert np.array_equal(wide[0][:rows, :2].cpu().numpy(), want[0]) and np.array_equal(wide[1][:rows, 1:].cpu().numpy(), want[1])
        assert bool((wide[0][:, 2] == 5).all()) and bool((wide[1][:, 0] == 5).all()) and bool((wide[:, rows] == 5).all())


def tolerance(spread, out, reach, lengths, dim, dt):
    """Half a step of the output's type, and twice (numerator and denominator) the
    weights' relative error: half a step of fp16; of the exponent, the fp32 sum of
    dim products (reach: the sum of their magnitudes), the factor's and the
    subtraction's roundings, each 2^-23 of at most reach + 16 (a whole last place:
    the matrix instruction's own rounding is not assumed to be to nearest), and
    exp2 to 2^-22;
    fp32 sums over the tokens.  Below that, fp16's least step: of a weight 2^-31 of
    the largest, of a value 2^-25 of the largest scale's unit."""
    exponent = 2.0 ** -23 * (dim + 8) * (reach[..., None] + 16)
    relative = 2.0 ** -11 + exponent + 2.0 ** -22 + 2.0 ** -23 * (lengths + 8)
    half_step = torch.finfo(dt).eps / 2
    return half_step * np.abs(out) + 2 * relative * spread * (1 + half_step) + torch.finfo(dt).tiny


def check_attention(q, codes, scales, pages, starts, lens, dt=None, **kw):
    rows, q_heads, dim = q.shape
    lse = torch.full((rows, q_heads), 3.0, device=DEV)
    dt = dt or q.dtype
    out = torch.full((rows, q_heads, dim), 9.0, dtype=dt, device=DEV)
    got = ops.attention_kv(q, gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens), lse=lse, out=out, **kw)
    assert got is out
    scale = kw.get("scale") or dim ** -0.5
    want, wlse, spread, reach = twin.attention(q.float().cpu().numpy(), codes, scales, pages, starts, lens, scale, kw.get("causal", True), kw.get("window", 0))
    inside = np.zeros(rows, bool)
    for _, row0, n, _, _ in twin.rows_of(starts, lens, pages.shape[1] * codes.shape[2] * 32, rows):
        inside[row0:row0 + n] = True
    got, lse = got.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert (got[~inside] == 9.0).all() and (lse[~inside] == 3.0).all()
    used = pages[(pages >= 0) & (pages < codes.shape[0])]
    biggest = 448.0 * 2.0 ** (scales[used][..., 1].max(initial=0) - 127.0)
    bound = tolerance(spread, want, reach, int(lens.max(initial=0)), dim, dt) + biggest * 2.0 ** -31 * max(1, int(lens.max(initial=0)))
    lost = np.isnan(want)
    assert (np.isnan(got) == lost)[inside].all()
    off = np.where(lost, 0.0, np.abs(got - want)) / np.where(lost, 1.0, bound)
    assert off[inside].max(initial=0.0) <= 1.0, off[inside].max()
    empty = np.isneginf(wlse)
    assert (np.isneginf(lse) == empty)[inside].all() and (got[inside][empty[inside]] == 0).all()
    step = 2.0 ** -11 + 2.0 ** -23 * (dim + 8) * (reach + 16) + 2.0 ** -22 * (np.abs(np.where(empty, 0, wlse)) + 16)
    fine = inside[:, None] & ~empty & ~np.isnan(wlse)
    assert (np.abs(lse - np.where(empty, 0, wlse)) <= step)[fine].all()
    assert np.isnan(lse[inside[:, None] & np.isnan(wlse)]).all()
    return got


# (page, heads, q heads, dim), (rows, tokens) of each sequence, (causal, window)
ATTENDS = [
    ((32, 1, 1, 64), [(1, 1)], (True, 0)),
    ((32, 2, 12, 256), [(1, 300)], (True, 0)),
    ((64, 2, 6, 128), [(1, 1), (1, 31), (1, 32), (1, 33), (1, 64), (1, 65), (1, 500), (0, 9)], (True, 0)),
    ((96, 4, 4, 64), [(1, 1100), (1, 2), (2, 700)], (True, 0)),
    ((64, 1, 20, 64), [(1, 3000)], (True, 0)),
    ((256, 1, 6, 256), [(16, 1500)], (True, 0)),
    ((32, 2, 10, 128), [(70, 70), (3, 90), (33, 161)], (True, 0)),
    ((64, 2, 2, 64), [(130, 700), (1, 1000)], (True, 0)),
    ((32, 2, 4, 128), [(40, 100), (5, 2), (2, 0)], (True, 0)),  # rows without a token
    ((32, 1, 7, 256), [(19, 45), (64, 64)], (False, 0)),
    ((64, 2, 8, 128), [(50, 400), (1, 900), (30, 30)], (True, 33)),
    ((64, 1, 3, 64), [(40, 600)], (False, 50)),
    ((32, 2, 2, 64), [(9, 70)], (True, 1)),
    ((32, 4, 16, 128), [(300, 900)], (True, 0)),
    ((64, 2, 12, 256), [(150, 600), (20, 20)], (True, 0)),
    ((32, 1, 71, 64), [(1, 500), (3, 77)], (True, 0)),  # more heads of a group than rows of a tile
    ((32, 1, 150, 128), [(1, 300), (7, 70)], (True, 60)),
]


@pytest.mark.parametrize("shape,seqs,mask", ATTENDS)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention(shape, seqs, mask, dt):
    page, heads, q_heads, dim = shape
    rng = np.random.default_rng([page, q_heads, dim, len(seqs)])
    per = [-(-t // page) for _, t in seqs]
    pool = sum(per) + 2
    codes, scales = filled(rng, pool, page, heads, dim)
    codes[..., 0, :] = rng.choice(codes.reshape(-1)[codes.reshape(-1) & 127 < 60], codes[..., 0, :].shape)  # keys mostly small
    pages = page_table(rng, per, pool, max(per) + 1)
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    lens = np.array([t for _, t in seqs], np.int32)
    wide = torch.from_numpy(rng.standard_normal((int(starts[-1]) + 1, q_heads + 1, dim))).to(DEV, TYPES[dt])
    check_attention(wide[:, 1:], codes, scales, pages, starts, lens, causal=mask[0], window=mask[1])
    check_attention(wide[:, 1:], codes, scales, pages, starts, lens, causal=mask[0], window=mask[1], scale=0.3,
                    dt=torch.float16 if dt == "bf16" else torch.bfloat16)


# the kernels of a call, and sizes for which it takes them: q heads, heads, (rows, tokens) of each
# sequence; pages of 64 tokens
PLANS = [
    ("stream 16", (2, 2, [(1, 90)])),
    ("stream 16 shared", (2, 2, [(1, 2755), (1, 0), (1, 77), (0, 900)])),
    ("stream 32", (6, 1, [(3, 90), (4, 64), (2, 33)])),
    ("stream 32 shared", (6, 1, [(3, 2600), (4, 1111)])),
    ("tile 64", (20, 1, [(2, 90), (40, 41)])),
    ("tile 64 split", (20, 1, [(2, 1300)])),
    ("tile 128", (64, 64, [(70, 96), (100, 100), (40, 90), (70, 71), (70, 95)])),
    ("tile 128 split", (20, 1, [(300, 2600)])),
    ("tile 256", (64, 64, [(300, 319), (260, 300), (333, 333)])),
    ("tile 256 split", (32, 4, [(513, 3200), (540, 999)])),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("plan,sizes", PLANS)
def test_every_plan(plan, sizes, dim):
    q_heads, heads, seqs = sizes
    rng = np.random.default_rng([dim, len(plan)])
    per = [-(-t // 64) for _, t in seqs]
    rows, pool = sum(n for n, _ in seqs), sum(per) + 1
    took = ops.attention_kv_plan(rows, len(seqs), q_heads, heads, dim, max(per) * 64)
    assert took.rstrip("0123456789").rstrip() == plan.rstrip("0123456789").rstrip() and took.split()[:2] == plan.split()[:2], took
    print(f"[gpu kv] {took}, D = {dim}", flush=True)
    codes, scales = filled(rng, pool, 64, heads, dim)
    codes[..., 0, :] = rng.choice(codes.reshape(-1)[codes.reshape(-1) & 127 < 60], codes[..., 0, :].shape)
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((rows, q_heads, dim))).to(DEV, torch.float16 if dim == 128 else torch.bfloat16)
    pages = page_table(rng, per, pool)
    check_attention(q, codes, scales, pages, starts, np.array([t for _, t in seqs], np.int32))
    if pages.shape[1] > 3:  # a hole, and a window that leaves workgroups without tokens
        pages[0, 1] = -1
        check_attention(q, codes, scales, pages, starts, np.array([t for _, t in seqs], np.int32), window=100, causal=dim != 64)


MIXED = [[(1, 2000), (1, 1), (70, 1400), (0, 300), (1, 700), (1, 2111), (100, 60), (2, 1999)],
         [(200, 2100)] + [(1, 100 + 150 * i) for i in range(14)]]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs", MIXED)
@pytest.mark.parametrize("mask", [(True, 0), (True, 70), (True, 1), (True, 1300), (False, 0), (False, 1300)])
def test_prompts_beside_single_tokens(seqs, mask, dim):
    """Sequences of many tiles among those of one, all shared by the same workgroups."""
    heads, group, page = 2, 1, 64
    rng = np.random.default_rng([dim, len(seqs)])
    per = [-(-t // page) for _, t in seqs]
    rows, pool = sum(n for n, _ in seqs), sum(per) + 1
    assert "stream" in ops.attention_kv_plan(rows, len(seqs), heads * group, heads, dim, max(per) * page)
    codes, scales = filled(rng, pool, page, heads, dim)
    codes[..., 0, :] = rng.choice(codes.reshape(-1)[codes.reshape(-1) & 127 < 60], codes[..., 0, :].shape)
    q = torch.from_numpy(rng.standard_normal((rows, heads * group, dim))).to(DEV, torch.bfloat16)
    check_attention(q, codes, scales, page_table(rng, per, pool), np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32),
                    np.array([t for _, t in seqs], np.int32), causal=mask[0], window=mask[1])


def small_case(seed=0, dt=torch.float16, dim=128, n=5, tokens=100, heads=2, group=3, page=32):
    rng = np.random.default_rng(seed)
    pool = -(-tokens // page) + 1
    codes, scales = filled(rng, pool, page, heads, dim)
    codes[..., 0, :] = rng.choice(codes.reshape(-1)[codes.reshape(-1) & 127 < 60], codes[..., 0, :].shape)
    pages = page_table(rng, [pool - 1], pool)
    q = torch.from_numpy(rng.standard_normal((n, heads * group, dim))).to(DEV, dt)
    return q, codes, scales, pages, np.array([0, n], np.int32), np.array([tokens], np.int32)


@pytest.mark.parametrize("n,dim", [(1, 256), (5, 128), (40, 64), (60, 256)])
def test_what_a_row_does_not_see_does_not_reach_it(n, dim):
    """NaN codes, and the largest scales, behind the last token; pages that are none,
    among them the whole of a sequence; a token of NaN seen by the later rows only."""
    q, codes, scales, pages, starts, lens = small_case(n=n, dim=dim)
    clean = check_attention(q, codes, scales, pages, starts, lens)
    for t in range(100, 128):
        place = [twin.bytes_of(kind, dim)[t % 32] for kind in (0, 1)]
        for kind in (0, 1):
            codes[pages[0, t // 32], :, 0, kind][:, place[kind]] = 127
    assert np.array_equal(check_attention(q, codes, scales, pages, starts, lens), clean)
    unused = next(p for p in range(codes.shape[0]) if p not in pages[0])
    codes[unused], scales[unused] = 255, 254
    gaps = pages.copy()
    gaps[0, 1], gaps[0, 2] = -1, codes.shape[0]
    check_attention(q, codes, scales, gaps, starts, lens)
    check_attention(q, codes, scales, np.full_like(pages, -5), starts, lens)
    if n > 1:  # the token of row n - 2 is lost: that row and the last see it
        t = 98
        codes[pages[0, t // 32], :, 0, 0][:, twin.bytes_of(0, dim)[t % 32]] = 127
        codes[pages[0, t // 32], :, 0, 1][:, twin.bytes_of(1, dim)[t % 32]] = 0
        lost = check_attention(q, codes, scales, pages, starts, lens)
        assert np.array_equal(lost[:n - 2], clean[:n - 2]) and np.isnan(lost[n - 2:]).all()


def test_scales_far_apart():
    """Blocks of values 2^40 apart, an empty (zero) block, keys whose scale differs."""
    for dim, n in ((64, 1), (128, 9), (256, 50)):
        q, codes, scales, pages, starts, lens = small_case(n=n, dim=dim, dt=torch.bfloat16)
        scales[pages[0, 0], :, 0, 1] = 80
        scales[pages[0, 2], :, 0, 1] = 126
        codes[pages[0, 1], :, 0, 1] = 0
        scales[pages[0, 1], :, 0, 1] = 0
        scales[pages[0, 1], 0, 0, 0] = 124
        check_attention(q, codes, scales, pages, starts, lens)
        scales[..., 1] = np.where(scales[..., 1] > 100, 3, 0)  # values of 2^-120
        check_attention(q, codes, scales, pages, starts, lens)


# q heads, heads, rows, tokens, window: which kernels run is test_every_plan's matter
UNSEEN = [(2, 2, 14, 100, 0), (2, 1, 16, 1284, 0), (6, 2, 5, 99, 32), (4, 1, 8, 2597, 31), (20, 1, 70, 99, 0),
          (20, 1, 40, 1300, 46), (64, 64, 70, 100, 0), (32, 4, 300, 999, 100),
          (1, 1, 700, 2600, 64), (20, 1, 300, 2600, 0), (32, 4, 530, 2000, 0)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,heads,rows,tokens,window", UNSEEN)
def test_values_that_only_other_rows_see(q_heads, heads, rows, tokens, window, dim):
    """The largest values in the last block, which the last rows alone see, and with a
    window in one that only the first do: not a bit changes in the others.  Of the
    scales 2^118 and 2^120, codes of 448 on the second are 2^128.8, past the 2^128 that
    fp32 and bf16 hold: the rows that see those have no value to compare with."""
    q, codes, scales, pages, starts, lens = small_case(n=rows, tokens=tokens, dim=dim, heads=heads, group=q_heads // heads, page=64,
                                                      dt=torch.bfloat16)
    args = dict(window=window)
    clean = check_attention(q, codes, scales, pages, starts, lens, **args)
    at = tokens - rows + np.arange(rows)
    last, first = (tokens - 1) // 32, max(tokens - rows - window + 1, 0) // 32
    same, edge = at < last * 32, bool(window) and first < last - 1
    if edge:
        same &= at - window >= first * 32 + 31
    assert same.any() and not same.all()
    for e in (118, 120):
        scales[pages[0, last // 2], :, last % 2, 1] = 127 + e
        if edge:
            scales[pages[0, first // 2], :, first % 2, 1] = 127 + e
        if e == 118:
            got = check_attention(q, codes, scales, pages, starts, lens, **args)
        else:
            got = ops.attention_kv(q, gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens), **args).float().cpu().numpy()
        assert np.array_equal(got[same], clean[same])


def test_queries_of_any_size():
    """Rows of zeros, of fp16's largest and least values, of an infinity and of NaN."""
    q, codes, scales, pages, starts, lens = small_case(n=6, dim=64)
    codes[..., 0, :] &= 0x87  # keys of the least codes
    q[0], q[1], q[2] = 0, q[1].sign() * 65504, q[2].sign() * 6e-8
    check_attention(q, codes, scales, pages, starts, lens)
    q[4, 1, 3], q[5] = math.nan, math.inf
    check_attention(q, codes, scales, pages, starts, lens)


def test_a_token_that_is_not_finite_is_lost_alone():
    rng = np.random.default_rng(2)
    heads, dim = 2, 128
    k, v = (rng.standard_normal((40, heads, dim)).astype(np.float32) for _ in range(2))
    k[3, 0, 7], k[9, 1, 0], v[20, 0, 127], v[21, 1, 5], v[39, 0, 1] = math.nan, math.inf, -math.inf, math.nan, 3e38
    codes, scales = filled(rng, 3, 32, heads, dim)
    pages, starts, lens = np.array([[2, 0]], np.int32), np.array([0, 40], np.int32), np.array([55], np.int32)
    c, s = gpu(codes), gpu(scales)
    assert ops.append_kv(gpu(k), gpu(v), c, s, gpu(pages), gpu(starts), gpu(lens)) is None
    twin.append(k, v, codes, scales, pages, starts, lens)
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes)
    q = torch.from_numpy(rng.standard_normal((40, 4, dim))).to(DEV, torch.bfloat16)
    out = check_attention(q, codes, scales, pages, starts, lens)
    assert [int(np.argmax(np.isnan(out[:, h, 0]))) for h in (0, 2)] == [3, 9]


def test_a_grid_that_grows_token_by_token():
    """Decode steps whose values grow and shrink: the older codes follow the grid."""
    rng = np.random.default_rng(3)
    heads, dim = 2, 64
    codes, scales = filled(rng, 4, 32, heads, dim)
    pages = np.array([[3, 1]], np.int32)
    c, s = gpu(codes), gpu(scales)
    for t in range(40):
        size = np.float32(2.0 ** ((t * 7) % 23 - 8))
        k, v = (size * rng.standard_normal((1, heads, dim)).astype(np.float32) for _ in range(2))
        starts, lens = np.array([0, 1], np.int32), np.array([t + 1], np.int32)
        ops.append_kv(gpu(k), gpu(v), c, s, gpu(pages), gpu(starts), gpu(lens))
        twin.append(k, v, codes, scales, pages, starts, lens)
        assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes), t


def test_values_at_the_borders_of_the_grid():
    """Ties and their neighbours, the largest code, subnormal codes, zeros of either sign."""
    dim, heads = 64, 1
    grid = twin._POSITIVE
    mid = (grid[:-1] + grid[1:]) / 2
    x = np.concatenate((grid, mid, np.nextafter(mid.astype(np.float32), np.float32(0)), np.nextafter(mid.astype(np.float32), np.float32(1e9)))).astype(np.float32)
    x = np.concatenate((x, -x, [448.0, 448.0]))
    for power in (0, -100, 60):
        flat = np.resize(np.ldexp(x, power).astype(np.float32), (64, heads, dim))
        flat[::32, :, 0] = np.float32(448 * 2.0 ** power)  # both blocks have the same grid
        codes, scales = np.zeros((2, heads, 1, 2, 32 * dim), np.uint8), np.zeros((2, heads, 1, 2), np.uint8)
        pages, starts, lens = np.array([[0, 1]], np.int32), np.array([0, 64], np.int32), np.array([64], np.int32)
        c, s = gpu(codes), gpu(scales)
        ops.append_kv(gpu(flat), gpu(flat[::-1]), c, s, gpu(pages), gpu(starts), gpu(lens))
        twin.append(flat, flat[::-1], codes, scales, pages, starts, lens)
        assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes)


def test_positions_outside_the_table():
    rng = np.random.default_rng(4)
    k = rng.standard_normal((4, 1, 64)).astype(np.float32)
    q = rng.standard_normal((4, 2, 64)).astype(np.float32)
    table, positions = rope_table(10, 32), np.array([3, 10, -1, 9], np.int32)
    codes, scales = np.zeros((1, 1, 1, 2, 2048), np.uint8), np.zeros((1, 1, 1, 2), np.uint8)
    pages, starts, lens = np.array([[0]], np.int32), np.array([0, 4], np.int32), np.array([4], np.int32)
    c, s = gpu(codes), gpu(scales)
    out = ops.append_kv(gpu(k), gpu(k), c, s, gpu(pages), gpu(starts), gpu(lens), q=gpu(q), rope=gpu(table), positions=gpu(positions))
    want = twin.append(k, k, codes, scales, pages, starts, lens, q=q, rope=table, positions=positions)
    assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scales)
    lost = torch.isnan(torch.from_numpy(want))
    assert torch.equal(torch.isnan(out.cpu()), lost) and torch.equal(out.cpu()[~lost], torch.from_numpy(want).bfloat16()[~lost])
    assert lost[1, :, :32].all() and not lost[1, :, 32:].any() and not lost[0].any()


def test_arrays_that_make_no_sense_stay_within_the_buffers():
    """starts that fall, lie outside the rows or are negative; lens past the pages."""
    rng = np.random.default_rng(6)
    q, codes, scales, pages, _, _ = small_case(n=8, dim=64)
    pages = np.repeat(pages, 3, 0)
    for starts, lens in (([5, 3, 9, 2], [10, 10, 10]), ([-4, 2, 100, 100], [1 << 30, -7, 5]), ([8, 8, 8, 8], [100, 100, 100])):
        check_attention(q, codes, scales, pages, np.array(starts, np.int32), np.array(lens, np.int32))
        k = torch.from_numpy(rng.standard_normal((8, 2, 64))).to(DEV, torch.float32)
        c, s = gpu(codes), gpu(scales)
        ops.append_kv(k, k, c, s, gpu(np.full_like(pages, 1 << 20)), ints(starts), ints(lens), q=k)
        assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scales)
        ops.read_kv(c, s, gpu(pages), ints(starts), ints(lens), 8)
    torch.cuda.synchronize()


def test_nothing_to_do():
    q, codes, scales, pages, starts, lens = small_case(n=2, dim=64)
    args = gpu(codes), gpu(scales), gpu(pages)
    assert ops.attention_kv(q[:0], *args, ints([0, 0]), gpu(lens)).shape == (0, 6, 64)
    none = gpu(pages)[:0], ints([0]), torch.empty(0, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 4)
    assert bool((ops.attention_kv(q, *args[:2], *none, out=out) == 4).all())
    no_pages = torch.empty((1, 0), dtype=torch.int32, device=DEV)
    assert bool((ops.attention_kv(q, *args[:2], no_pages, gpu(starts), gpu(lens)) == 0).all())
    k, v = ops.read_kv(*args[:2], no_pages, gpu(starts), gpu(lens), 2)
    assert not bool(k.any()) and not bool(v.any())


@pytest.mark.parametrize("plan,sizes", PLANS)
def test_a_cache_without_pages(plan, sizes):
    """Every sequence's entries name pages, of a pool that has none: rows see nothing."""
    q_heads, heads, seqs = sizes
    rng = np.random.default_rng(len(plan))
    codes, scales = ops.new_kv_cache(0, 64, heads, 128, DEV)
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    lens = np.array([t for _, t in seqs], np.int32)
    pages = np.zeros((len(seqs), -(-int(lens.max()) // 64)), np.int32)
    q = torch.from_numpy(rng.standard_normal((int(starts[-1]), q_heads, 128))).to(DEV, torch.bfloat16)
    print(f"[gpu kv] no pages, {plan}", flush=True)
    for causal in (True, False):
        check_attention(q, codes.cpu().numpy(), scales.cpu().numpy(), pages, starts, lens, causal=causal)
    k = torch.ones((len(q), heads, 128), device=DEV)
    assert torch.equal(ops.append_kv(k, k, codes, scales, gpu(pages), gpu(starts), gpu(lens), q=k), k.bfloat16())
    back = ops.read_kv(codes, scales, gpu(pages), gpu(starts), gpu(lens), len(q))
    assert not back[0].any() and not back[1].any()


def test_in_place():
    q, codes, scales, pages, starts, lens = small_case(n=40, dim=128, tokens=700)
    cache = gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens)
    want = ops.attention_kv(q, *cache)
    got = q.clone()
    assert ops.attention_kv(got, *cache, out=got) is got and torch.equal(got, want)
    packed = torch.randn(40, 10, 128, device=DEV).half()
    rope = gpu(rope_table(700, 64))
    mine = packed.clone()
    want = ops.append_kv(packed[:, 6:8], packed[:, 8:], *cache, q=packed[:, :6], rope=rope, dtype=torch.float16)
    ops.append_kv(mine[:, 6:8], mine[:, 8:], *cache, q=mine[:, :6], rope=rope, q_out=mine[:, :6])
    assert torch.equal(mine[:, :6], want) and torch.equal(mine[:, 6:], packed[:, 6:])


def test_rows_at_any_element():
    """Heads and rows that begin at odd elements, heads outside rows."""
    rng = np.random.default_rng(12)
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        flat = torch.from_numpy(rng.standard_normal(1 + 9 * 5 * 67)).to(DEV, dt)
        odd = flat[1:].view(9, 5, 67)[:, :, 1:65]  # strides 335 and 67
        codes, scales = filled(rng, 3, 32, 1, 64)
        pages, starts, lens = np.array([[2, 0]], np.int32), np.array([0, 9], np.int32), np.array([40], np.int32)
        c, s = gpu(codes), gpu(scales)
        out = torch.zeros(1 + 3 * 9 * 65, dtype=torch.float16, device=DEV)[1:].view(3, 9, 65).transpose(0, 1)[:, :, :64]  # heads outside rows
        ops.append_kv(odd[:, 3:4], odd[:, 4:], c, s, gpu(pages), gpu(starts), gpu(lens), q=odd[:, :3], q_out=out, rope=gpu(rope_table(50, 48)))
        host = odd.float().cpu().numpy()
        want = twin.append(host[:, 3:4], host[:, 4:], codes, scales, pages, starts, lens, q=host[:, :3], rope=rope_table(50, 48))
        assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scales)
        assert torch.equal(out.cpu(), torch.from_numpy(want).half())
        if dt != torch.float32:
            check_attention(odd[:, :3], codes, scales, pages, starts, lens)
            near = ops.attention_kv(out, c, s, gpu(pages), gpu(starts), gpu(lens))
            assert torch.equal(ops.attention_kv(out, c, s, gpu(pages), gpu(starts), gpu(lens), out=torch.zeros_like(odd[:, :3], dtype=dt).half()), near)


def test_offsets_past_32_bits():
    """A page that begins past 4 GB of the pool, and rows past 4 GB of the queries' buffer."""
    dim, heads, page = 256, 8, 256
    pool = 4200  # of 1 MB
    codes, scales = ops.new_kv_cache(pool, page, heads, dim, DEV)
    rng = np.random.default_rng(8)
    k, v = (torch.from_numpy(rng.standard_normal((300, heads, dim))).to(DEV, torch.float32) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((3, heads, dim))).to(DEV, torch.float16)
    near = ops.new_kv_cache(2, page, heads, dim, DEV)
    far = codes, scales, ints([[pool - 1, pool - 2]])
    near = *near, ints([[1, 0]])
    for cache in (near, far):
        ops.append_kv(k, v, *cache, ints([0, 300]), ints([300]))
    want = ops.attention_kv(q, *near, ints([0, 3]), ints([300]))
    assert torch.equal(ops.attention_kv(q, *far, ints([0, 3]), ints([300])), want)
    for a, b in zip(ops.read_kv(*near, ints([0, 300]), ints([300]), 300), ops.read_kv(*far, ints([0, 300]), ints([300]), 300)):
        assert torch.equal(a, b)
    del codes, scales, far
    stride = (1 << 30) // dim * dim
    wide = torch.empty(2 * stride + heads * dim, dtype=torch.float16, device=DEV).as_strided((3, heads, dim), (stride, dim, 1))
    wide.copy_(q)
    assert torch.equal(ops.attention_kv(wide, *near, ints([0, 3]), ints([300]), out=wide), want)


def test_graph_replays_with_other_lengths():
    """A captured decode step (append, attention): lengths and pages change between replays."""
    dim, heads, q_heads, page, seqs = 128, 2, 8, 32, 3
    rng = np.random.default_rng(9)
    codes, scales = ops.new_kv_cache(3 * 40, page, heads, dim, DEV)
    eager = codes.clone(), scales.clone()
    pages, starts = gpu(page_table(rng, [40] * seqs, 3 * 40)), ints(list(range(seqs + 1)))
    lens = ints([1, 1, 1])
    x = torch.zeros(seqs, q_heads + 2 * heads, dim, device=DEV)
    rope = gpu(rope_table(1300, dim))

    def step(c, s):
        q = ops.append_kv(x[:, q_heads:q_heads + heads], x[:, q_heads + heads:], c, s, pages, starts, lens, q=x[:, :q_heads], rope=rope)
        return ops.attention_kv(q, c, s, pages, starts, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(codes, scales)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(codes, scales)
    step(*eager)
    codes.copy_(eager[0]), scales.copy_(eager[1])
    for i in range(6):
        lens.copy_(ints([1 + i, 200 * i + 7, 1280 - i]))
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape)))
        graph.replay()
        want = step(*eager)
        assert torch.equal(out, want) and torch.equal(codes, eager[0]) and torch.equal(scales, eager[1]), i
        torch.cuda.synchronize()


def test_calls_on_two_streams():
    """The current stream of the tensors' device is used; calls with workspaces of their own overlap."""
    q, codes, scales, pages, starts, lens = small_case(n=1, dim=256, tokens=6000)
    cache = gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens)
    want = ops.attention_kv(q, *cache)
    need = ops.attention_kv_workspace_bytes(1, 1, 6, 2, 256, pages.shape[1] * 32)
    assert need > 0
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(ops.attention_kv(q, *cache, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


def test_a_prompt_in_pieces_equals_the_prompt_at_once():
    """Micro-batches (append, attention) leave the same cache where blocks are whole, and each row's
    attention within its tolerance; then the layer's products read the result."""
    dim, heads, q_heads, page, n = 128, 2, 6, 64, 256
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(n, (q_heads + 2 * heads) * dim, device=DEV, generator=g).view(n, -1, dim)
    rope, w = gpu(rope_table(n, dim)), 1 + 0.1 * torch.randn(dim, device=DEV, generator=g)

    def layer(sizes):
        codes, scales = ops.new_kv_cache(4, page, heads, dim, DEV)
        pages, out, at = ints([[2, 0, 3, 1]]), [], 0
        for size in sizes:
            y = x[at:at + size]
            at += size
            q = ops.append_kv(y[:, q_heads:q_heads + heads], y[:, q_heads + heads:], codes, scales, pages, ints([0, size]), ints([at]),
                              q=y[:, :q_heads], rope=rope, q_weight=w, k_weight=w, dtype=torch.float16)
            out.append(ops.attention_kv(q, codes, scales, pages, ints([0, size]), ints([at])))
        return torch.cat(out), codes, scales

    (a, *cache_a), (b, *cache_b) = layer([n]), layer([96, 32, 128])
    assert all(torch.equal(x, y) for x, y in zip(cache_a, cache_b))
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -11 * float(a.float().abs().max())
    weights = torch.randn(64, q_heads * dim, device=DEV, generator=g)
    act, s = ops.quantize_mx4(a.view(n, -1))
    y = ops.gemm_mx4(ops.prepare_weights_mx4(weights), act, s, 64, q_heads * dim)
    exact = a.view(n, -1).double() @ weights.double().t()
    assert float((y - exact).norm() / exact.norm()) < 0.25  # 4-bit rows and weights: half a step of 2^-2 each, at most

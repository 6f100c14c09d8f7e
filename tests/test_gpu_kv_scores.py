"""Attention over the 8-bit cache where scores, or the scales of keys and values,
leave the ordinary range: on the GPU, against the definition in 64 bits (kv_twin),
by every plan."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_twin as twin  # noqa: E402
from hadamard_rotated_w4a4_amd import ops  # noqa: E402
from test_gpu_kv import DEV, PLANS, filled, gpu, page_table, tolerance  # noqa: E402

pytestmark = pytest.mark.gpu


def plan_case(plan, sizes, dim, seed):
    """A batch that takes the plan: (rng, sequences, page table, codes, scales, starts, lens)."""
    q_heads, heads, seqs = sizes
    rng = np.random.default_rng([dim, len(plan), seed])
    per = [-(-t // 64) for _, t in seqs]
    rows, pool = sum(n for n, _ in seqs), sum(per) + 1
    took = ops.attention_kv_plan(rows, len(seqs), q_heads, heads, dim, max(per) * 64)
    assert took.rstrip("0123456789").rstrip() == plan.rstrip("0123456789").rstrip() and took.split()[:2] == plan.split()[:2], took
    codes, scales = filled(rng, pool, 64, heads, dim)
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    return rng, page_table(rng, per, pool), codes, scales, starts, np.array([t for _, t in seqs], np.int32)


def run(q, codes, scales, pages, starts, lens, **kw):
    lse = torch.full(q.shape[:2], 3.0, device=DEV)
    out = ops.attention_kv(q, gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens), lse=lse, **kw)
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def off(lse, wlse):
    return np.abs(np.where(np.isneginf(wlse), 0.0, lse) - np.where(np.isneginf(wlse), 0.0, wlse))


def put(codes, kind, values, dim):
    """E4M3 codes [pages, heads, blocks, 32 tokens, dim] into a pool's keys (0) or values (1)."""
    codes[:, :, :, kind][..., twin.bytes_of(kind, dim).reshape(-1)] = values.reshape(*values.shape[:3], -1)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("plan,sizes", PLANS)
def test_the_largest_scores(plan, sizes, dim):
    """Queries of +-65504 (fp16; 65280 in bf16) and keys of +-448 on scales of 2^0 to 2^8:
    scores up to 2^41, that every step holds exactly.  A key has n of its channels, the
    others are zero, with one pattern of signs for all: a score is n 2^e times one number
    (two products of which have 22 bits with n), so scores are either equal, or 10^6
    apart where a last place is 2^18 at most.  A row is the mean of the values of its
    largest scores, all with one weight: errors are the sums' and the weight's alone."""
    q_heads, heads, _ = sizes
    rng, pages, codes, scales, starts, lens = plan_case(plan, sizes, dim, 1)
    dt, most = (torch.float16, 65504.0) if dim == 128 else (torch.bfloat16, 65280.0)
    signs = rng.choice([-1.0, 1.0], dim)
    scales[..., 0] = rng.integers(127, 136, scales[..., 0].shape)
    channels = rng.integers(0, dim + 1, (*codes.shape[:3], 32, 1))
    sign = rng.choice([-1.0, 1.0], channels.shape) * signs
    put(codes, 0, np.where(np.arange(dim) < channels, np.where(sign < 0, 0xFE, 0x7E), 0).astype(np.uint8), dim)
    rows = int(starts[-1])
    q = torch.from_numpy(most * signs * rng.choice([-1.0, 1.0], (rows, q_heads, 1))).to(DEV, dt)
    want, wlse, spread, reach = twin.attention(q.float().cpu().numpy(), codes, scales, pages, starts, lens, dim ** -0.5)
    got, lse = run(q, codes, scales, pages, starts, lens)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tolerance(spread, want, 0 * reach, int(lens.max()), dim, dt)).all()
    # the factor's rounding, the product's, of log2 e to e back: 2^-24 each of the score, and a last place
    some = ~np.isneginf(wlse)
    assert (np.isneginf(lse) == ~some).all()
    assert (off(lse, wlse)[some] <= 2.0 ** -11 + 2.0 ** -21 * (np.abs(wlse[some]) + 16)).all()


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40])
def test_large_scores_of_any_kind(size):
    """Ordinary keys, and queries that make scores of 2^15 to 2^43: rounding decides
    between near scores, but a row is a mean of values that it sees, and its lse its
    largest score, to the rounding of a score (dim products and five operations)."""
    for plan, sizes in PLANS:
        q_heads, heads, _ = sizes
        rng, pages, codes, scales, starts, lens = plan_case(plan, sizes, 64, 2)
        rows = int(starts[-1])
        q = torch.from_numpy(size * rng.standard_normal((rows, q_heads, 64))).to(DEV, torch.bfloat16)
        want, wlse, _, reach = twin.attention(q.float().cpu().numpy(), codes, scales, pages, starts, lens, 0.125)
        got, lse = run(q, codes, scales, pages, starts, lens)
        some = ~np.isneginf(wlse)
        most = 448.0 * 2.0 ** (scales[..., 1].max() - 127.0)
        assert np.isfinite(got).all() and np.abs(got).max() <= most * (1 + 2.0 ** -8), plan
        assert (np.isneginf(lse) == ~some).all(), plan
        # within a rounding of the largest, a score more: at most all of the tokens
        assert (off(lse, wlse)[some] <= 2.0 ** -23 * (64 + 8) * reach[some] + np.log(lens.max()) + 1).all(), plan


# code of a key's first channel (times a query's 8, over sqrt(dim): 62 to 68, or 20 to 22), for each dim
FAR, NEAR = {64: 64.0, 128: 96.0, 256: 128.0}, {64: 20.0, 128: 30.0, 256: 44.0}


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("plan,sizes", PLANS)
@pytest.mark.parametrize("first,power", [(FAR, 30), (NEAR, 30), (FAR, -30)], ids=["no weight", "their share", "all the weight"])
def test_blocks_of_other_value_scales(first, power, plan, sizes, dim):
    """A third of a sequence's blocks have values 2^30 times the others', and weights of
    e^-62 and less, or of about e^-21 (2^-30: what they add is of the others' size); or
    2^-30 of the others' size and all the weight.  What counts keeps its bits: what a token
    adds is off by 2^-24 at most of the largest scale times its block's largest weight, and
    not of the largest scale."""
    q_heads, heads, seqs = sizes
    rng, pages, codes, scales, starts, lens = plan_case(plan, sizes, dim, 3)
    dt = torch.float16 if dim == 128 else torch.bfloat16
    keys = rng.choice(np.arange(256)[np.arange(256) & 127 < 60], (*codes.shape[:3], 32, dim)).astype(np.uint8)
    keys[..., 0] = 0
    put(codes, 0, keys, dim)
    plain = codes.copy()  # the same without what sets blocks apart: what roundings of scores are measured by
    chosen = np.full(len(seqs), 1 << 30)  # a sequence's first such block
    sign = -1 if power > 0 else 1
    code = int(np.argmin(np.abs(twin.E4M3[:127] - first[dim]))) | (128 if sign < 0 else 0)
    for b, (_, tokens) in enumerate(seqs):
        for blk in range(1, -(-tokens // 32)):
            if rng.random() < 0.34:
                at = pages[b, blk // 2], slice(None), blk % 2
                keys[at][..., 0] = code
                only = keys[at].copy()
                only[..., 1:] = 0
                codes[at][:, 0][:, twin.bytes_of(0, dim).reshape(-1)] = only.reshape(heads, -1)
                scales[at] = np.array([127, int(scales[at][0, 1]) + power], np.uint8)
                chosen[b] = min(chosen[b], blk)
    rows = int(starts[-1])
    queries = rng.standard_normal((rows, q_heads, dim))
    queries[..., 0] = 8.0
    q = torch.from_numpy(queries).to(DEV, dt)
    exact = q.float().cpu().numpy()
    want, wlse, spread, _ = twin.attention(exact, codes, scales, pages, starts, lens, dim ** -0.5)
    reach = twin.attention(exact, plain, np.where(scales == 127, 122, scales), pages, starts, lens, dim ** -0.5)[3]
    got, lse = run(q, codes, scales, pages, starts, lens)
    s = sign * first[dim] * 8 * dim ** -0.5
    unit = np.zeros((rows, 1, 1))  # the largest scale times its block's largest weight, of each row
    for b, row0, n, at, _ in twin.rows_of(starts, lens, pages.shape[1] * 64, rows):
        sees = np.arange(at, at + n) >= 32 * chosen[b]
        unit[row0:row0 + n, 0, 0] = np.where(sees, max(2.0 ** -5 * np.exp(min(-s, 0)), 2.0 ** (power - 5) * np.exp(min(s, 0))) * np.e, 2.0 ** -5)
    bound = tolerance(spread, want, reach, int(lens.max()), dim, dt) + 448 * unit * 2.0 ** -24 * int(lens.max())
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()
    some = ~np.isneginf(wlse)
    assert (np.isneginf(lse) == ~some).all()
    step = 2.0 ** -11 + 2.0 ** -23 * (dim + 8) * (reach + abs(s) + 16) + 2.0 ** -22 * (np.abs(np.where(some, wlse, 0)) + 16)
    assert (off(lse, wlse) <= step)[some].all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("plan,sizes", PLANS)
def test_factors_past_fp32s_normal_range(plan, sizes, dim):
    """A block's key scale times the call's scale below 2^-126, under bf16 queries of 2^122
    (scores of about 0.1, 2^-127 a key); past 2^128, where queries of zeros still see every
    token alike; and a scale that fp32 has only zero for."""
    q_heads, heads, _ = sizes
    rng, pages, codes, scales, starts, lens = plan_case(plan, sizes, dim, 4)
    keys = rng.choice(np.arange(256)[np.arange(256) & 127 < 60], (*codes.shape[:3], 32, dim)).astype(np.uint8)
    put(codes, 0, keys, dim)
    rows, length = int(starts[-1]), int(lens.max())
    ordinary = rng.standard_normal((rows, q_heads, dim))
    for queries, key_scales, scale in ((ordinary * 2.0 ** 122, (0, 3), dim ** -0.5), (0 * ordinary, (240, 247), 1e5), (ordinary, (100, 127), 1e-60)):
        scales[..., 0] = rng.integers(*key_scales, scales[..., 0].shape)
        q = torch.from_numpy(queries).to(DEV, torch.bfloat16)
        want, wlse, spread, reach = twin.attention(q.float().cpu().numpy(), codes, scales, pages, starts, lens, scale)
        got, lse = run(q, codes, scales, pages, starts, lens, scale=scale)
        bound = tolerance(spread, want, reach, length, dim, torch.bfloat16) + 448 * 2.0 ** -5 * 2.0 ** -24 * length
        assert (np.abs(got - want) <= bound).all(), (scale, (np.abs(got - want) / bound).max())
        some = ~np.isneginf(wlse)
        assert (np.isneginf(lse) == ~some).all()
        assert (off(lse, wlse) <= 2.0 ** -11 + 2.0 ** -23 * (dim + 8) * (reach + 16) + 2.0 ** -22 * (np.abs(np.where(some, wlse, 0)) + 16))[some].all()

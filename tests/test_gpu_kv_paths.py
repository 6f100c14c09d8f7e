"""The key/value cache and its attention on paths that only longer, wider or more
numerous calls take, on the GPU, against the definitions written a second time
(kv_twin)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_twin as twin  # noqa: E402
from hadamard_rotated_w4a4_amd import ops  # noqa: E402
from test_gpu_kv import DEV, PLANS, check_attention, filled, gpu, ints, page_table, rope_table  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def whole_pools(monkeypatch):
    """kv_twin's token_values from a pool decoded once: long sequences take seconds otherwise."""
    made = {}

    def values(codes, scales, pages, b, token, kind):
        key = (id(codes), id(scales), kind)
        if key not in made:
            place = twin.bytes_of(kind, codes.shape[4] // 32)
            unit = 2.0 ** (scales[..., kind].astype(np.float64) - 127)
            made[key] = codes, scales, twin.E4M3[codes[:, :, :, kind][..., place]] * unit[..., None, None]
        blk = token // 32
        page = int(pages[b, blk // codes.shape[2]])
        return made[key][2][page, :, blk % codes.shape[2], token % 32] if 0 <= page < codes.shape[0] else None

    monkeypatch.setattr(twin, "token_values", values)


def case(seed, heads, group, dim, seqs, width=None, page=64, dt=torch.bfloat16):
    """(q, codes, scales, page table, starts, lens) of sequences of (rows, tokens)."""
    rng = np.random.default_rng(seed)
    per = [-(-t // page) for _, t in seqs]
    pool = sum(per) + 1
    codes, scales = filled(rng, pool, page, heads, dim)
    codes[..., 0, :] = rng.choice(codes.reshape(-1)[codes.reshape(-1) & 127 < 60], codes[..., 0, :].shape)  # keys mostly small
    starts = np.cumsum([0] + [n for n, _ in seqs]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(starts[-1]), heads * group, dim))).to(DEV, dt)
    return q, codes, scales, page_table(rng, per, pool, width), starts, np.array([t for _, t in seqs], np.int32)


def plan_of(q, codes, pages, window=0):
    return ops.attention_kv_plan(q.shape[0], len(pages), q.shape[1], codes.shape[1], q.shape[2], pages.shape[1] * codes.shape[2] * 32, window)


def alike(took, plan):
    """The kernels of the plan, whatever the number of workgroups or splits."""
    return took.split()[:2] == plan.split()[:2] and ("shared" in took, "split" in took) == ("shared" in plan, "split" in plan)


def spoilt(q, codes, pages):
    need = ops.attention_kv_workspace_bytes(q.shape[0], len(pages), q.shape[1], codes.shape[1], q.shape[2], pages.shape[1] * codes.shape[2] * 32)
    return torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN, and indexes of -1


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("plan,sizes", PLANS)
def test_missing_pages_under_every_plan(plan, sizes, dim):
    """Single holes, a stretch of a sequence's middle, all but its last page, and every
    page: in a workspace of NaN, so that nothing that no one wrote is taken."""
    q_heads, heads, seqs = sizes
    q, codes, scales, pages, starts, lens = case([dim, len(plan), 5], heads, q_heads // heads, dim, seqs, dt=torch.float16 if dim == 128 else torch.bfloat16)
    assert alike(plan_of(q, codes, pages), plan)
    own = -(-int(lens[0]) // 64)
    rng = np.random.default_rng(dim)
    for holes in (rng.random(own) < 0.3, (np.arange(own) >= own // 3) & (np.arange(own) < own - 1), np.arange(own) < own - 1, np.arange(own) >= 0):
        some = pages.copy()
        some[0, :own][holes] = rng.choice([-1, codes.shape[0], 1 << 30], int(holes.sum()))
        check_attention(q, codes, scales, some, starts, lens, causal=dim != 64, workspace=spoilt(q, codes, some))


# plans, sizes for which a call with the window takes them
WINDOWS = [
    ("stream 16 shared", (2, 1, [(1, 5900), (1, 0), (1, 4077), (0, 900), (1, 5000)]), 4500),
    ("stream 32 shared", (1, 6, [(3, 5600), (4, 4111)]), 4000),
    ("tile 64 split", (1, 20, [(2, 1300)]), 1000),
    ("tile 128 split", (1, 20, [(300, 2600)]), 2000),
    ("tile 256 split", (4, 8, [(513, 3200), (540, 999)]), 2600),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("plan,sizes,window", WINDOWS)
def test_windows_under_plans_that_share_tokens(plan, sizes, window, dim):
    heads, group, seqs = sizes
    q, codes, scales, pages, starts, lens = case([dim, len(plan), 6], heads, group, dim, seqs)
    assert alike(plan_of(q, codes, pages, window), plan)
    for causal in (True, False):
        check_attention(q, codes, scales, pages, starts, lens, causal=causal, window=window, workspace=spoilt(q, codes, pages))


def test_a_windows_plan_takes_no_more_workspace():
    """A call with a window is given what the sizes alone ask for, and runs in it."""
    for heads, group, dim, seqs in ((1, 20, 128, [(300, 2600)]), (2, 1, 256, [(1, 5900), (1, 77)]), (4, 2, 64, [(70, 700), (1, 1500)])):
        q, codes, scales, pages, starts, lens = case(dim, heads, group, dim, seqs)
        for window in (1, 70, 1000, 2400):
            check_attention(q, codes, scales, pages, starts, lens, window=window, workspace=spoilt(q, codes, pages))


def many(seqs, rows, long, at, short=45):
    """`seqs` sequences of `rows` rows, those of `at` of `long` tokens, the others of about
    `short`, and some without rows."""
    rng = np.random.default_rng(seqs)
    out = []
    for i in range(seqs):
        n = 0 if i % 16 == 5 or i == seqs - 2 else rows
        out.append((n, long - i % 7 if i in at else max(n, short + int(rng.integers(0, 40)))))
    return out


# plan, (heads, group, dim), (sequences, rows of each): unsplit beside so many, so that a
# workgroup has all 140 of a long sequence's blocks, or a half to a fifth of them
LONG = [
    ("tile 64", (2, 1, 64), (65, 40)), ("tile 128", (4, 6, 64), (64, 13)), ("tile 64", (1, 6, 128), (64, 13)), ("tile 128", (2, 6, 128), (66, 13)),
    ("tile 256", (2, 6, 128), (65, 40)), ("tile 64", (1, 6, 256), (64, 13)), ("tile 128", (2, 6, 256), (65, 13)),
    ("tile 64 split", (1, 1, 64), (64, 40)), ("tile 64 split", (1, 1, 128), (65, 40)), ("tile 64 split", (1, 1, 256), (66, 40)), ("tile 128 split", (1, 6, 128), (64, 90)),
]


@pytest.mark.parametrize("plan,heads,seqs", LONG)
def test_many_sequences_and_long_ones_in_tiles(plan, heads, seqs):
    """More than two times 64 blocks of one workgroup (addresses and scales are fetched 64
    blocks at a time), or more than 64 of two, in sequences on both sides of the 64th."""
    sizes = many(*seqs, 4480, (0, 31, seqs[0] - 1))
    q, codes, scales, pages, starts, lens = case([*heads, 7], *heads, sizes)
    took = plan_of(q, codes, pages)
    assert alike(took, plan), took
    print(f"[gpu kv] {took}, D = {heads[2]}", flush=True)
    check_attention(q, codes, scales, pages, starts, lens, workspace=spoilt(q, codes, pages))
    check_attention(q, codes, scales, pages, starts, lens, causal=False, window=4200)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs,heads,group,rows", [(80, 8, 1, 1), (130, 8, 2, 1), (65, 8, 4, 5)])
def test_long_sequences_streamed_by_one_workgroup(seqs, heads, group, rows, dim):
    """More than 32 steps of a wave (8192 tokens of a workgroup)."""
    q, codes, scales, pages, starts, lens = case([dim, seqs, 8], heads, group, dim, many(seqs, rows, 9000, (3, seqs - 1)), 256)
    assert alike(plan_of(q, codes, pages), "stream 16" if rows * group <= 16 else "stream 32")
    check_attention(q, codes, scales, pages, starts, lens)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs", [64, 65, 130])
@pytest.mark.parametrize("plan,group,rows", [("stream 16", 2, 1), ("stream 32", 6, 4), ("tile", 20, 4)])
def test_many_short_sequences(plan, group, rows, seqs, dim):
    q, codes, scales, pages, starts, lens = case([dim, seqs, 9], 1, group, dim, many(seqs, rows, 60, (0, 63)), 5)
    assert plan_of(q, codes, pages).startswith(plan)
    check_attention(q, codes, scales, pages, starts, lens, workspace=spoilt(q, codes, pages))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs,heads,group,rows", [(64, 1, 20, 1), (65, 1, 6, 3), (130, 2, 6, 1)])
def test_many_sequences_shared(seqs, heads, group, rows, dim):
    """Steps of more than 64 sequences summed, and tiles of the last ones joined."""
    sizes = many(seqs, rows, 2048, (0, 40, 62, 63, seqs - 1))
    q, codes, scales, pages, starts, lens = case([dim, seqs, 10], heads, group, dim, sizes)
    took = plan_of(q, codes, pages)
    if (seqs, dim) != (130, 64) and (seqs, dim) != (130, 128):
        assert "shared" in took, took
    check_attention(q, codes, scales, pages, starts, lens, workspace=spoilt(q, codes, pages))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sizes", [[(16, 8192)], [(16, 8192), (3, 50)], [(3, 70), (16, 8100)]])
def test_more_than_eight_splits(sizes, dim):
    """A verify block: splits joined by four waves a row, some of them empty for a short sequence."""
    q, codes, scales, pages, starts, lens = case([dim, len(sizes), 11], 1, 6, dim, sizes)
    took = plan_of(q, codes, pages)
    assert took.startswith("tile 64 split") and int(took.split()[3]) > 8, took
    check_attention(q, codes, scales, pages, starts, lens, workspace=spoilt(q, codes, pages))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,heads,group,tokens", [(256, 2, 4, 2500), (512, 4, 6, 700), (600, 1, 8, 700), (256, 1, 20, 600), (1, 2, 6, 300), (20, 1, 2, 500)])
def test_page_tables_wider_than_the_sequence(rows, heads, group, tokens, dim):
    """As a captured step has them: planned for 131072 tokens (many splits or workers),
    of which most are behind the end; entries there name no page, or any."""
    q, codes, scales, pages, starts, lens = case([dim, rows, 12], heads, group, dim, [(rows, tokens)], 2048)
    took = plan_of(q, codes, pages)
    assert "split" in took or "shared" in took, took
    print(f"[gpu kv] {took}, D = {dim}", flush=True)
    want = check_attention(q, codes, scales, pages, starts, lens, workspace=spoilt(q, codes, pages))
    pages[0, -(-tokens // 64):] = np.resize([0, 5, codes.shape[0], -9], 2048 - -(-tokens // 64))
    got = ops.attention_kv(q, gpu(codes), gpu(scales), gpu(pages), gpu(starts), gpu(lens), workspace=spoilt(q, codes, pages))
    assert np.array_equal(got.float().cpu().numpy(), want)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs", [64, 65, 130, 200])
def test_append_and_read_back_of_many_sequences(seqs, dim):
    """Rows and blocks of sequences past the 64th and 128th, some without rows."""
    rng = np.random.default_rng([seqs, dim])
    heads, q_heads, page = 2, 3, 32
    sizes = [(0 if i % 16 == 5 or i in (64, seqs - 2) else int(rng.integers(1, 5)), int(rng.integers(4, 90))) for i in range(seqs)]
    per = [-(-t // page) for _, t in sizes]
    pool = sum(per) + 1
    codes, scales = filled(rng, pool, page, heads, dim)
    pages = page_table(rng, per, pool)
    starts = np.cumsum([0] + [n for n, _ in sizes]).astype(np.int32)
    lens = np.array([t for _, t in sizes], np.int32)
    rows = int(starts[-1])
    x = rng.standard_normal((rows, q_heads + 2 * heads, dim)).astype(np.float32)
    q, k, v = x[:, :q_heads], x[:, q_heads:q_heads + heads], x[:, q_heads + heads:]
    rope = rope_table(100, 32)
    c, s, xs = gpu(codes), gpu(scales), gpu(x)
    on_gpu = gpu(pages), gpu(starts), gpu(lens)
    out = ops.append_kv(xs[:, q_heads:q_heads + heads], xs[:, q_heads + heads:], c, s, *on_gpu, q=xs[:, :q_heads], rope=gpu(rope), dtype=torch.float16)
    want = twin.append(k, v, codes, scales, pages, starts, lens, q=q, rope=rope)
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(c.cpu().numpy(), codes)
    assert torch.equal(out.cpu(), torch.from_numpy(want).half())
    exact = twin.read(codes, scales, pages, starts, lens, rows)
    for got, values in zip(ops.read_kv(c, s, *on_gpu, rows, dtype=torch.float32), exact):
        assert np.array_equal(got.cpu().numpy(), values)


def turned(x, weight, rope, at):
    """twin.turn of [rows, heads, dim] at once: the same fp32 operations, halves apart."""
    f = np.float32
    root = (1.0 / np.sqrt((x.astype(np.float64) ** 2).sum(2) / x.shape[2] + 1e-6)).astype(f)
    x = x * root[..., None] * weight
    half = rope.shape[1] // 2
    c, s = rope[at, None, :half], rope[at, None, half:]
    out = x.copy()
    out[..., :half] = x[..., :half] * c - x[..., half:2 * half] * s
    out[..., half:2 * half] = x[..., half:2 * half] * c + x[..., :half] * s
    return out


@pytest.mark.parametrize("rows,q_heads,dim,width", [(1500, 30, 128, 96), (1500, 31, 128, 128), (1200, 17, 256, 64), (3000, 70, 64, 64)])
def test_queries_in_several_passes(rows, q_heads, dim, width):
    """Rows so many that a wave takes heads in more than four passes (its loads run four ahead),
    the last group of heads not full; into a new output and in place."""
    rng = np.random.default_rng([rows, dim])
    step = 512 // dim
    passes = min(-(-q_heads // step), 8, rows * -(-q_heads // step) // 2048)
    assert passes > 4 and q_heads % (passes * step)
    x = (rng.standard_normal((rows, q_heads + 2, dim)) * np.exp(rng.standard_normal((rows, 1, 1)))).astype(np.float16)
    w = (1 + 0.1 * rng.standard_normal(dim)).astype(np.float32)
    rope, at = rope_table(4000, width), rng.integers(0, 4000, rows)
    turn = turned(x[:, :q_heads].astype(np.float32), w, rope, at)
    for row, head in ((0, 0), (rows - 1, q_heads - 1), (rows // 2, 5)):  # the two ways of writing it down
        assert np.array_equal(turn[row, head], twin.turn(x[row, head].astype(np.float32), w, 1e-6, rope, False, [int(at[row])] * (width // 2)))
    want = torch.from_numpy(turn).half()
    codes, scales = ops.new_kv_cache(-(-rows // 32), 32, 1, dim, DEV)
    pages = torch.arange(len(codes), dtype=torch.int32, device=DEV)[None]
    args = codes, scales, pages, ints([0, rows]), ints([rows])
    given = dict(rope=gpu(rope), positions=gpu(at.astype(np.int32)), q_weight=gpu(w))
    xs = gpu(x)
    assert torch.equal(ops.append_kv(xs[:, -2:-1], xs[:, -1:], *args, q=xs[:, :q_heads], dtype=torch.float16, **given).cpu(), want)
    ops.append_kv(xs[:, -2:-1], xs[:, -1:], *args, q=xs[:, :q_heads], q_out=xs[:, :q_heads], **given)
    assert torch.equal(xs[:, :q_heads].cpu(), want)

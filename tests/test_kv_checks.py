"""Refusals of the key/value cache's calls, without a GPU: the C ABI on fake
pointers (never dereferenced), the binding on CPU tensors."""
import ctypes
from ctypes import POINTER, Structure, byref, c_int, c_int64, c_void_p

import pytest

torch = pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import ops  # noqa: E402
from hadamard_rotated_w4a4_amd._lib import W4A4Error  # noqa: E402

OK, INVALID, KMUL, MISALIGNED, DTYPE, WS, HIP = range(7)
F32, F16, BF16 = range(3)
A, ODD = 0x10000000, 0x10000001


class Cache(Structure):
    _fields_ = [("codes", c_void_p), ("scales", c_void_p), ("pages", c_int64), ("page", c_int64), ("heads", c_int64), ("dim", c_int64)]


class Batch(Structure):
    _fields_ = [("pages", c_void_p), ("ld", c_int64), ("pages_per_seq", c_int64), ("starts", c_void_p), ("lens", c_void_p),
                ("seqs", c_int64), ("rows", c_int64)]


class Heads(Structure):
    _fields_ = [("data", c_void_p), ("row_stride", c_int64), ("head_stride", c_int64)]


class Rope(Structure):
    _fields_ = [("table", c_void_p), ("table_rows", c_int64), ("width", c_int64), ("positions", c_void_p), ("ld", c_int64),
                ("axes", c_void_p), ("n_axes", c_int64), ("interleaved", c_int)]


@pytest.fixture(scope="module")
def L():
    return ops.lib()


def made(cls, base, **changes):
    return cls(**{**base, **changes})


CACHE = dict(codes=A, scales=A, pages=10, page=64, heads=4, dim=128)
BATCH = dict(pages=A, ld=5, pages_per_seq=5, starts=A, lens=A, seqs=2, rows=7)
ROPE = dict(table=A, table_rows=100, width=64, positions=None, ld=0, axes=None, n_axes=1, interleaved=0)
NOTHING = dict(rows=0)  # calls that would be launched if they were taken: none here is


def append(L, dt=BF16, odt=F16, q_heads=8, eps=1e-6, k=A, v=A, q=A, out=A + 4096, strides=(2048, 128), weight=A, cache={}, batch={}, rope={}, out_strides=(1024, 128)):
    c, b = made(Cache, CACHE, **cache), made(Batch, BATCH, **batch)
    r = None if rope is None else made(Rope, ROPE, **rope)
    return L.w4a4_append_kv(dt, byref(Heads(k, *strides)), byref(Heads(v, *strides)), byref(Heads(q, *strides)), q_heads,
                            byref(Heads(out, *out_strides)), odt, c_void_p(weight), c_void_p(weight), eps,
                            None if r is None else byref(r), byref(c), byref(b), None)


def attend(L, dt=BF16, odt=F16, q_heads=8, q=A, out=A + 4096, lse=None, ld=8, scale=0.1, window=0, cache={}, batch={}, ws=A, nbytes=None, strides=(1024, 128)):
    c, b = made(Cache, CACHE, **cache), made(Batch, BATCH, **batch)
    need = L.w4a4_attention_kv_workspace_bytes(b.rows, b.seqs, q_heads, c.heads, c.dim, b.pages_per_seq * c.page)
    return L.w4a4_attention_kv(byref(Heads(q, *strides)), dt, q_heads, byref(Heads(out, *strides)), odt, c_void_p(lse), ld, scale, 1, window,
                               byref(c), byref(b), c_void_p(ws), need if nbytes is None else nbytes, None)


def read(L, dt=BF16, k=A, v=A, strides=(512, 128), cache={}, batch={}):
    c, b = made(Cache, CACHE, **cache), made(Batch, BATCH, **batch)
    return L.w4a4_read_kv(byref(c), byref(b), dt, byref(Heads(k, *strides)), byref(Heads(v, *strides)), None)


BAD_CACHES = [dict(dim=96), dict(dim=512), dict(page=48), dict(page=0), dict(heads=0), dict(heads=8193), dict(pages=-1),
              dict(pages=1 << 31), dict(pages=1 << 28, heads=4, page=64), dict(page=(1 << 30) + 32)]
BAD_BATCHES = [dict(seqs=-1), dict(seqs=65537), dict(rows=-1), dict(rows=2097121), dict(ld=4), dict(pages_per_seq=-1),
               dict(pages_per_seq=(1 << 24) + 1, ld=1 << 26), dict(ld=1 << 31)]
NULLS = [dict(pages=None), dict(starts=None), dict(lens=None)]


def test_size_queries(L):
    assert L.w4a4_kv_cache_code_bytes(10, 64, 4, 128) == 10 * 64 * 4 * 128 * 2
    assert L.w4a4_kv_cache_scale_bytes(10, 64, 4, 128) == 10 * 2 * 4 * 2
    for bad in ((10, 48, 4, 128), (10, 64, 0, 128), (10, 64, 4, 100), (-1, 64, 4, 128)):
        assert L.w4a4_kv_cache_code_bytes(*bad) == L.w4a4_kv_cache_scale_bytes(*bad) == 0
    query = L.w4a4_attention_kv_workspace_bytes
    assert query(1, 1, 24, 4, 256, 1 << 17) > 0
    assert query(1, 1, 24, 4, 256, 256) == 0  # few tokens: nothing to share
    for bad in ((-1, 1, 24, 4, 256, 100), (1, 1, 23, 4, 256, 1 << 17), (1, 1, 2, 4, 256, 1 << 17), (1, 1, 24, 4, 250, 1 << 17),
                (1, 1, 24, 4, 256, (1 << 30) + 1), (2097121, 1, 24, 4, 256, 1 << 17), (1, 65537, 24, 4, 256, 1 << 17)):
        assert query(*bad) == 0


def test_attention_plan(L):
    sizes = (512, 1, 24, 4, 256, 32768)
    whole = ops.attention_kv_plan(*sizes)
    assert whole.startswith("tile 256 split ") and ops.attention_kv_plan(*sizes, 64).startswith("tile ")
    query = L.w4a4_attention_kv_plan
    assert query(*sizes, 0, None, 99) == len(whole)
    text = ctypes.create_string_buffer(b"left", 8)
    assert query(*sizes, 0, text, 5) == len(whole) and text.value == b"tile"
    for bad in ((0, 1, 24, 4, 256, 100, 0), (1, 0, 24, 4, 256, 100, 0), (1, 1, 23, 4, 256, 100, 0), (1, 1, 24, 4, 255, 100, 0),
                (1, 1, 24, 4, 256, -1, 0), (1, 1, 24, 4, 256, 100, -1)):
        assert query(*bad, text, 8) == 0 and text.value == b""
    # a window never takes more workspace than the sizes alone
    for tokens in (500, 3000, 40000):
        assert ops.attention_kv_plan(300, 2, 24, 4, 128, tokens, 1) != ""


@pytest.mark.parametrize("call", [append, attend, read])
def test_sizes_are_refused_and_nothing_to_do_is_fine(L, call):
    for bad in BAD_CACHES:
        assert call(L, cache=bad) == INVALID, bad
        assert call(L, cache=bad, batch=NOTHING) == INVALID, bad
    for bad in BAD_BATCHES:
        assert call(L, batch=bad) == INVALID, bad
    for bad in NULLS:
        assert call(L, batch=bad) == INVALID, bad
    for bad in (dict(codes=None), dict(scales=None)):
        assert call(L, cache=bad) == INVALID, bad
    assert call(L, cache=dict(codes=A + 8)) == MISALIGNED
    assert call(L, cache=dict(scales=ODD)) == MISALIGNED
    for name in ("pages", "starts", "lens"):
        assert call(L, batch={name: A + 2}) == MISALIGNED
    assert call(L, batch=dict(rows=0)) == OK and call(L, batch=dict(seqs=0)) == OK
    assert call(L, dt=3) == DTYPE and call(L, dt=-1) == DTYPE


def test_append_refusals(L):
    for bad in (dict(k=None), dict(v=None), dict(q=None), dict(out=None), dict(strides=(-1, 128)), dict(strides=(2048, -128)),
                dict(out_strides=(1000, 128)), dict(out_strides=(1024, 100)), dict(out_strides=(64, 128)), dict(q_heads=0), dict(q_heads=8193),
                dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(out=A, odt=BF16), dict(out=A, odt=F16)):
        assert append(L, **bad) == INVALID, bad
    for bad in (dict(width=0), dict(width=24), dict(width=144), dict(table_rows=-1), dict(table=None), dict(n_axes=2), dict(axes=A),
                dict(axes=A, positions=A, n_axes=0), dict(axes=A, positions=A, n_axes=3, ld=6), dict(table_rows=1 << 31)):
        assert append(L, rope=bad) == INVALID, bad
    assert append(L, odt=F32) == DTYPE and append(L, odt=7) == DTYPE
    for bad in (dict(k=ODD), dict(v=ODD), dict(q=ODD), dict(out=ODD), dict(weight=A + 2), dict(rope=dict(table=A + 2)),
                dict(rope=dict(positions=A + 1)), dict(dt=F32, k=A + 2)):
        assert append(L, **bad) == MISALIGNED, bad
    assert append(L, eps=0.0, weight=None, batch=NOTHING) == OK
    # nothing is launched where the grid would not fit
    assert append(L, q_heads=8192, batch=dict(rows=2097120)) == INVALID


def test_positions_of_no_axis_are_refused(L):
    """As with axes: every pair would turn by NaN."""
    for n in (0, -1):
        assert append(L, rope=dict(positions=A, n_axes=n)) == INVALID
    assert append(L, rope=dict(positions=A, n_axes=1), batch=NOTHING) == OK and append(L, rope=dict(n_axes=0), batch=NOTHING) == OK


def test_attention_refusals(L):
    long = dict(pages_per_seq=4096, ld=4096)
    for bad in (dict(q=None), dict(out=None), dict(q_heads=6), dict(q_heads=0), dict(q_heads=2), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=1e60), dict(scale=3e38), dict(window=-1), dict(lse=A, ld=7), dict(strides=(-1, 128)), dict(strides=(1024, 64)),
                dict(out=A), dict(batch=long, ws=None)):
        assert attend(L, **bad) == INVALID, bad
    assert attend(L, dt=F32) == DTYPE and attend(L, odt=F32) == DTYPE
    for bad in (dict(q=ODD), dict(out=ODD), dict(lse=A + 2), dict(batch=long, ws=A + 128)):
        assert attend(L, **bad) == MISALIGNED, bad
    assert attend(L, batch=long, nbytes=1 << 10) == WS
    assert attend(L, q_heads=8192, cache=dict(heads=1), batch=dict(rows=2097120), strides=(1 << 20, 128)) == INVALID


def test_read_refusals(L):
    for bad in (dict(k=None), dict(v=None), dict(strides=(500, 128)), dict(strides=(512, 64)), dict(strides=(-512, 128))):
        assert read(L, **bad) == INVALID, bad
    assert read(L, k=ODD) == MISALIGNED and read(L, dt=F32, v=A + 2) == MISALIGNED


def tensors(rows=4, heads=2, q_heads=4, dim=64, seqs=2):
    i = dict(dtype=torch.int32)
    return dict(k=torch.zeros(rows, heads, dim), v=torch.zeros(rows, heads, dim), codes=torch.zeros(3, heads, 2, 2, 32 * dim, dtype=torch.uint8),
                scales=torch.zeros(3, heads, 2, 2, dtype=torch.uint8), pages=torch.zeros(seqs, 3, **i), starts=torch.zeros(seqs + 1, **i),
                lens=torch.zeros(seqs, **i)), torch.zeros(rows, q_heads, dim)


def test_binding_refusals():
    base, q = tensors()
    half = q.half()
    bytes_ = dict(dtype=torch.uint8)

    def refused(call, text, *more, without=(), **changes):
        args = {**{n: x for n, x in base.items() if n not in without}, **changes}
        with pytest.raises(W4A4Error, match=text):
            call(*more, **args)

    common = [("codes: expected", dict(codes=torch.zeros(3, 2, 2, 2048, **bytes_))), ("codes: dtype", dict(codes=torch.zeros(3, 2, 2, 2, 2048))),
              ("heads of 32", dict(codes=torch.zeros(3, 2, 2, 2, 1024, **bytes_))), ("scales: expected", dict(scales=torch.zeros(3, 2, 1, 2, **bytes_))),
              ("pages: dtype", dict(pages=torch.zeros(2, 3, dtype=torch.int64))), ("pages must be", dict(pages=torch.zeros(3, dtype=torch.int32))),
              ("pages: strides", dict(pages=torch.zeros(3, 2, dtype=torch.int32).t())), ("starts: 8 bytes", dict(starts=torch.zeros(2, dtype=torch.int32))),
              ("lens: dtype", dict(lens=torch.zeros(2))), ("codes is required", dict(codes=None))]
    kv = ("k", "v")
    for text, change in common + [("live on the GPU", {})]:
        refused(ops.append_kv, text, **change)
        refused(ops.attention_kv, text, half, without=kv, **change)
        refused(ops.read_kv, text, without=kv, rows=4, **change)
    for text, change in [("k: expected", dict(k=q[0])), ("k: shape", dict(k=q)), ("v: shape", dict(v=base["v"][:3])), ("one dtype", dict(v=base["v"].half())),
                         ("one dtype", dict(q=half)), ("q: shape", dict(q=q[:2])), ("unit stride", dict(v=torch.zeros(4, 64, 2).transpose(1, 2))),
                         ("q_out without q", dict(q_out=half)), ("q_out: dtype", dict(q=q, dtype=torch.float32)), ("q_out: shape", dict(q=q, q_out=half[:3])),
                         ("expected a torch.dtype", dict(q=q, dtype="half")), ("q_weight: ", dict(q_weight=torch.ones(63))),
                         ("eps", dict(k_weight=torch.ones(64), eps=0.0)), ("rope: expected", dict(rope=torch.zeros(9, 24))),
                         ("rope: expected", dict(rope=torch.zeros(9, 80))), ("rope: dtype", dict(rope=torch.zeros(9, 32, dtype=torch.float64))),
                         ("positions: expected", dict(rope=torch.zeros(9, 32), positions=torch.zeros(3, dtype=torch.int32))),
                         ("positions: dtype", dict(rope=torch.zeros(9, 32), positions=torch.zeros(4, dtype=torch.int64))),
                         ("need axes", dict(rope=torch.zeros(9, 32), positions=torch.zeros(3, 4, dtype=torch.int32))),
                         ("axes: 15 bytes", dict(rope=torch.zeros(9, 32), positions=torch.zeros(3, 4, dtype=torch.int32), axes=torch.zeros(15, **bytes_))),
                         ("axes without", dict(rope=torch.zeros(9, 32), axes=torch.zeros(16, **bytes_))),
                         ("need rope", dict(positions=torch.zeros(4, dtype=torch.int32)))]:
        refused(ops.append_kv, text, **change)
    for text, x, change in [("q: dtype", q, {}), ("q: expected", half[0], {}), ("query heads", half[:, :3], {}), ("q: shape", half[:, :, :32], {}),
                            ("scale", half, dict(scale=0.0)), ("window", half, dict(window=-1)), ("out: dtype", half, dict(out=q)),
                            ("out: shape", half, dict(out=half[:3])), ("lse: expected float32", half, dict(lse=half[:, :, 0])),
                            ("lse: shape", half, dict(lse=torch.zeros(4, 3))), ("workspace", half, dict(pages=torch.zeros(2, 999, dtype=torch.int32), workspace=torch.zeros(9, **bytes_)))]:
        refused(ops.attention_kv, text, x, without=kv, **change)
    refused(ops.read_kv, "negative", without=kv, rows=-1)
    refused(ops.read_kv, "one dtype", without=kv, rows=4, k=base["k"], v=base["v"].half())
    refused(ops.read_kv, "k: shape", without=kv, rows=5, k=base["k"])
    with pytest.raises(W4A4Error, match="no cache"):
        ops.new_kv_cache(3, 40, 2, 64, "cpu")
    assert [tuple(x.shape) for x in ops.new_kv_cache(3, 64, 2, 64, "cpu")] == [(3, 2, 2, 2, 2048), (3, 2, 2, 2)]

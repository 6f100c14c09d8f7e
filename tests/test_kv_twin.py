"""Pins of the key/value cache's second implementation (kv_twin): to PyTorch's
E4M3, to closed forms, to a dense softmax."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_twin as twin  # noqa: E402


def test_codes_are_pytorchs():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(twin.E4M3, every, equal_nan=True)
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(1 << 18) * np.exp(3 * rng.standard_normal(1 << 18))).clip(-448, 448).astype(np.float32)
    grid = twin._POSITIVE
    x = np.concatenate((x, grid, -grid, (grid[:-1] + grid[1:]) / 2)).astype(np.float32)  # values, ties
    assert np.array_equal(twin.e4m3_codes(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_byte_of_a_block_has_one_code(dim):
    for kind in (0, 1):
        assert np.array_equal(np.sort(twin.bytes_of(kind, dim).reshape(-1)), np.arange(32 * dim))


def test_exponents():
    for e in (-127, -100, 0, 77):
        top = 448.0 * 2.0 ** e
        assert twin.exponent(top) == e
        assert twin.exponent(np.nextafter(top, np.inf)) == e + 1
        if e > -127:
            assert twin.exponent(np.nextafter(top / 2, 0.0)) == e - 1
    assert twin.exponent(0.0) == twin.exponent(1e-45) == -127


def test_rotations_turn_by_the_tables_angle():
    rng = np.random.default_rng(1)
    x = rng.standard_normal(64).astype(np.float32)
    angle = rng.uniform(0, 6, (5, 16))
    table = np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32)
    for interleaved in (False, True):
        y = twin.turn(x, None, 0.0, table, interleaved, [i % 5 for i in range(16)])
        for i in range(16):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 16)
            z = complex(x[a], x[b]) * np.exp(1j * angle[i % 5, i])
            assert abs(complex(y[a], y[b]) - z) <= 4 * 2.0 ** -24 * abs(z) + 2.0 ** -23 * abs(z)
        assert np.array_equal(y[32:], x[32:])
    w = rng.standard_normal(64).astype(np.float32)
    y = twin.turn(x, w, 1e-6, None, False, None).astype(np.float64)
    exact = x.astype(np.float64) / math.sqrt((x.astype(np.float64) ** 2).mean() + 1e-6) * w
    assert (np.abs(y - exact) <= 3 * 2.0 ** -24 * np.abs(exact)).all()


def test_what_is_appended_is_read_and_attended():
    """Values on the grid come back as they were; attention is the dense softmax of them."""
    rng = np.random.default_rng(2)
    heads, dim, n = 2, 64, 50
    k, v = (rng.integers(-8, 9, (n, heads, dim)).astype(np.float32) / 4 for _ in range(2))
    codes, scales = np.full((3, heads, 1, 2, 32 * dim), 255, np.uint8), np.zeros((3, heads, 1, 2), np.uint8)
    pages, starts, lens = np.array([[2, 0]], np.int32), np.array([0, n], np.int32), np.array([n], np.int32)
    twin.append(k, v, codes, scales, pages, starts, lens)
    assert np.array_equal(twin.read(codes, scales, pages, starts, lens, n), np.stack((k, v)))
    q = rng.standard_normal((n, 2 * heads, dim))
    out, lse, _, _ = twin.attention(q, codes, scales, pages, starts, lens, 0.1, window=7)
    at = np.arange(n)
    hidden = (at[None] > at[:, None]) | (at[None] <= at[:, None] - 7)
    for h in range(2 * heads):
        s = torch.from_numpy(0.1 * q[:, h] @ k[:, h // 2].T.astype(np.float64)).masked_fill(torch.from_numpy(hidden), -math.inf)
        assert np.allclose(out[:, h], torch.softmax(s, 1).numpy() @ v[:, h // 2].astype(np.float64), rtol=1e-12, atol=1e-12)
        assert np.allclose(lse[:, h], torch.logsumexp(s, 1).numpy(), rtol=1e-12)

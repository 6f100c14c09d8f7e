"""The key/value cache and the attention over it, written a second time from the
definitions in include/w4a4.h: numpy, byte by byte, attention in 64 bits."""
import math

import numpy as np


def _e4m3_table():
    out = np.zeros(256)
    for c in range(256):
        size, fraction = c >> 3 & 15, c & 7
        value = (8 + fraction) * 2.0 ** (size - 10) if size else fraction * 2.0 ** -9
        out[c] = math.nan if c & 127 == 127 else (-value if c & 128 else value)
    return out


E4M3 = _e4m3_table()
_POSITIVE = E4M3[:127]  # ascending


def e4m3_codes(x):
    """Codes of float values (|x| <= 448), to nearest, ties to the even code."""
    a = np.abs(x.astype(np.float64))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    low, high = _POSITIVE[hi - 1], _POSITIVE[hi]
    up = (a - low > high - a) | ((a - low == high - a) & (hi % 2 == 0))
    return np.where(up, hi, hi - 1).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)


def key_byte(t, d):
    return d // 32 * 1024 + d // 16 % 2 * 512 + t * 16 + d % 16


def value_byte(t, d):
    return d // 32 * 1024 + t // 4 % 2 * 512 + d % 32 * 16 + t // 8 % 2 * 8 + t // 16 * 4 + t % 4


_T = np.arange(32)[:, None]


def bytes_of(kind, dim):
    """[32 tokens, dim]: where a code lies in the keys' (0) or values' (1) bytes of a block."""
    d = np.arange(dim)[None]
    return key_byte(_T, d) if kind == 0 else value_byte(_T, d)


def rows_of(starts, lens, per_seq_tokens, rows):
    """(sequence, first row, rows, token of the first row, tokens), as the arrays mean."""
    out = []
    for b in range(len(lens)):
        lo = min(max(int(starts[b]), 0), rows)
        hi = min(max(int(starts[b + 1]), lo), rows)
        length = min(max(int(lens[b]), 0), per_seq_tokens)
        out.append((b, lo, hi - lo, length - (hi - lo), length))
    return out


def exponent(top):
    """The least e >= -127 with top <= 448 * 2^e."""
    e = -127
    if top > 0:
        e = max(-127, math.frexp(top)[1] - 12)
        while top > 448.0 * 2.0 ** e:
            e += 1
        while e > -127 and top <= 448.0 * 2.0 ** (e - 1):
            e -= 1
    return e


def turn(x, weight, eps, rope, interleaved, at):
    """One head's row (float32 [dim]) normed and turned; at: position of each pair."""
    f = np.float32
    with np.errstate(invalid="ignore", over="ignore"):
        if weight is not None:
            root = f(1.0 / math.sqrt(float((x.astype(np.float64) ** 2).sum()) / len(x) + eps)) if np.isfinite(x).all() else f(np.nan)
            x = x * root * weight
        if rope is None:
            return x
        half = rope.shape[1] // 2
        c, s = np.full(half, np.nan, f), np.full(half, np.nan, f)
        for i in range(half):
            if 0 <= at[i] < rope.shape[0]:
                c[i], s[i] = rope[at[i], i], rope[at[i], half + i]
        one, two = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
        out = x.copy()
        out[one] = x[one] * c - x[two] * s
        out[two] = x[two] * c + x[one] * s
        return out


def position_of(row, token, rope, positions, axes):
    half = rope.shape[1] // 2
    if positions is None:
        return [token] * half
    if axes is None:
        return [int(positions.reshape(-1)[row])] * half
    p = positions.reshape(-1, positions.shape[-1])
    return [int(p[axes[i], row]) if axes[i] < p.shape[0] else -1 for i in range(half)]


def append(k, v, codes, scales, pages, starts, lens, q=None, rope=None, positions=None, axes=None, interleaved=False,
           q_weight=None, k_weight=None, eps=1e-6):
    """float32 arrays [rows, heads, dim]; codes and scales are changed in place;
    returns q turned, in float32 (rows outside every sequence as they came)."""
    n_pages, heads, per_page, _, width = codes.shape
    dim, rows = width // 32, k.shape[0]
    out = None if q is None else q.copy()
    for b, row0, n, first, length in rows_of(starts, lens, pages.shape[1] * per_page * 32, rows):
        at = [None if rope is None else position_of(row0 + i, first + i, rope, positions, axes) for i in range(n)]
        if q is not None:
            for i in range(n):
                for h in range(q.shape[1]):
                    out[row0 + i, h] = turn(q[row0 + i, h], q_weight, eps, rope, interleaved, at[i])
        for blk in range(max(first, 0) // 32, (length + 31) // 32 if n else 0):
            page = int(pages[b, blk // per_page])
            if not 0 <= page < n_pages:
                continue
            new = [t for t in range(max(first - 32 * blk, 0), min(length - 32 * blk, 32)) if 32 * blk + t >= first]
            kept = max(first - 32 * blk, 0)
            for h in range(heads):
                ks = [turn(k[row0 + 32 * blk + t - first, h], k_weight, eps, rope, interleaved, at[32 * blk + t - first]) for t in new]
                vs = [v[row0 + 32 * blk + t - first, h] for t in new]
                fine = [bool(np.isfinite(x).all() and np.isfinite(y).all()) for x, y in zip(ks, vs)]
                for kind, xs in ((0, ks), (1, vs)):
                    place, cell = bytes_of(kind, dim), codes[page, h, blk % per_page, kind]
                    e = exponent(max([float(np.abs(x).max()) for x, ok in zip(xs, fine) if ok], default=0.0))
                    was = int(scales[page, h, blk % per_page, kind]) - 127
                    if kept and was >= e:
                        e = was
                    elif kept:
                        for t in range(kept):
                            old = cell[place[t]]
                            cell[place[t]] = np.where(old & 127 == 127, old, e4m3_codes(np.nan_to_num(E4M3[old]) * 2.0 ** (was - e)) | (old & 128))
                    for t, x, ok in zip(new, xs, fine):
                        cell[place[t]] = e4m3_codes(np.ldexp(x.astype(np.float64), -e)) if ok else (127 if kind == 0 else 0)
                    scales[page, h, blk % per_page, kind] = e + 127
    return out


def token_values(codes, scales, pages, b, token, kind):
    """[heads, dim] in 64 bits; None where the token has no page."""
    n_pages, heads, per_page, _, width = codes.shape
    blk = token // 32
    page = int(pages[b, blk // per_page])
    if not 0 <= page < n_pages:
        return None
    place = bytes_of(kind, width // 32)[token % 32]
    unit = 2.0 ** (scales[page, :, blk % per_page, kind].astype(np.float64) - 127)
    return E4M3[codes[page, :, blk % per_page, kind][:, place]] * unit[:, None]


def read(codes, scales, pages, starts, lens, rows):
    heads, dim = codes.shape[1], codes.shape[4] // 32
    out = np.full((2, rows, heads, dim), np.nan)
    for b, row0, n, first, _ in rows_of(starts, lens, pages.shape[1] * codes.shape[2] * 32, rows):
        for i in range(n):
            for kind in (0, 1):
                x = token_values(codes, scales, pages, b, first + i, kind) if first + i >= 0 else None
                out[kind, row0 + i] = 0.0 if x is None else x
    return out


def attention(q, codes, scales, pages, starts, lens, scale, causal=True, window=0):
    """(out, lse, spread, reach): spread is sum p |v| / sum p, reach the largest
    sum |q k| * scale of a row: what errors are measured by.  float64."""
    n_pages, heads, per_page, _, width = codes.shape
    rows, q_heads, dim = q.shape
    group = q_heads // heads
    out, spread = np.zeros((rows, q_heads, dim)), np.zeros((rows, q_heads, dim))
    lse, reach = np.full((rows, q_heads), -np.inf), np.zeros((rows, q_heads))
    q = q.astype(np.float64)
    for b, row0, n, first, length in rows_of(starts, lens, pages.shape[1] * per_page * 32, rows):
        tokens = [t for t in range(length) if 0 <= int(pages[b, t // 32 // per_page]) < n_pages]
        if not tokens or not n:
            continue
        k = np.stack([token_values(codes, scales, pages, b, t, 0) for t in tokens], 1)  # [heads, tokens, dim]
        v = np.stack([token_values(codes, scales, pages, b, t, 1) for t in tokens], 1)
        j, at = np.array(tokens)[None], first + np.arange(n)[:, None]
        seen = np.ones((n, len(tokens)), bool)
        if causal:
            seen &= j <= at
        if window:
            seen &= j > at - window
        for h in range(q_heads):
            qs, kh, vh = q[row0:row0 + n, h], k[h // group], v[h // group]
            with np.errstate(invalid="ignore"):
                s = np.where(seen, scale * (qs @ kh.T), -np.inf)
                a = np.where(seen, scale * (np.abs(qs) @ np.abs(kh).T), 0.0)
            top = s.max(1, keepdims=True)
            p = np.where(seen, np.exp(s - np.where(np.isneginf(top), 0.0, top)), 0.0)
            total = p.sum(1)
            some = ~(total == 0)
            safe = np.where(some, total, 1.0)[:, None]
            out[row0:row0 + n, h] = np.where(some[:, None], p @ vh / safe, 0.0)
            spread[row0:row0 + n, h] = p @ np.abs(vh) / safe
            with np.errstate(divide="ignore"):
                lse[row0:row0 + n, h] = np.where(some, top[:, 0] + np.log(safe[:, 0]), -np.inf)
            reach[row0:row0 + n, h] = a.max(1)
    return out, lse, spread, reach

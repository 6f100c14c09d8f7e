"""Plain implementations of the quantised-row producers and the MXFP4 product,
on the CPU: 64-bit floating point where the definition has an exact value
(sums, the activation function, products), single fp32 operations where it
has a rounding.  Nothing here is shared with the kernels."""
import math

import numpy as np
import torch

C32 = np.float32(1.0 / math.sqrt(32.0))
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rounded(x64, dtype):
    """fp32 or fp64 array rounded to a torch dtype, as float32 (exact)."""
    return torch.from_numpy(np.ascontiguousarray(x64)).to(dtype).float().numpy()


def butterflies(v):
    """[..., 32] fp32: the unnormalised transform, stages 1, 2, 4, 8, 16."""
    v = v.astype(np.float32).copy()
    for h in (1, 2, 4, 8, 16):
        p = v.reshape(*v.shape[:-1], 32 // (2 * h), 2, h)
        a, b = p[..., 0, :].copy(), p[..., 1, :].copy()
        p[..., 0, :], p[..., 1, :] = a + b, a - b
    return v


def int_rows(v, top):
    """Rotated blocks on the int4 (top 7) or int8 (127) grid: integer codes
    [m, k] and fp32 scales [m, k/32]."""
    u = butterflies(v.reshape(v.shape[0], -1, 32))
    d = np.abs(u).max(-1) / np.float32(top)
    live = d >= np.float32(1.17549435e-38)
    inv = np.where(live, np.float32(1) / np.where(live, d, np.float32(1)), np.float32(0))
    t = u * inv[..., None]
    q = np.where(t < 0, -np.floor(-t.astype(np.float64) + 0.5), np.floor(t.astype(np.float64) + 0.5))
    q = np.clip(q, -top, top).astype(np.int8)
    return q.reshape(v.shape), np.where(live, d * C32, np.float32(0)).astype(np.float32)


def int4_bytes(q):
    """Byte 16 b + j of a row: element 32 b + j low, 32 b + j + 16 high."""
    b = q.reshape(q.shape[0], -1, 2, 16).astype(np.uint8) & 15
    return (b[:, :, 0] | b[:, :, 1] << 4).reshape(q.shape[0], -1)


def stride(k):
    return -(-(k // 32) // 8) * 8


def mx4_rows(v, rotate):
    """MXFP4 rows of fp32 v [m, k]: code bytes [m, k/2], scale bytes
    [m, stride] (padding 127).  Nearest by distance in 64 bits, ties to the
    even code."""
    with np.errstate(all="ignore"):
        b = v.astype(np.float32).reshape(v.shape[0], -1, 32)
        if rotate:
            b = butterflies(b) * C32
        finite = np.isfinite(b).all(-1)
        x = np.where(finite[..., None], b, np.float32(0)).astype(np.float64)
        top = np.abs(x).max(-1)
        e = np.where(top > 0, np.floor(np.frexp(np.where(top > 0, top, 1.0))[1] - 1.0) - 2, -127).clip(-127, 127).astype(int)
        a = np.minimum(np.ldexp(np.abs(x), -e[..., None]), 6.0)
        code = np.zeros(a.shape, np.uint8)
        best = np.abs(a - GRID[0])
        for i in range(1, 8):
            dist = np.abs(a - GRID[i])
            take = (dist < best) | ((dist == best) & (i % 2 == 0))
            code, best = np.where(take, np.uint8(i), code), np.minimum(best, dist)
        code = np.where(finite[..., None], code | np.where(np.signbit(b), 8, 0).astype(np.uint8), 0).astype(np.uint8)
    code = code.reshape(v.shape[0], -1, 2)
    scales = np.full((v.shape[0], stride(v.shape[1])), 127, np.uint8)
    scales[:, :v.shape[1] // 32] = np.where(finite, e + 127, 255)
    return (code[..., 0] | code[..., 1] << 4).astype(np.uint8), scales


def mx4_values(codes, scales, k):
    """MXFP4 rows as fp64 values (NaN blocks included)."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], k // 32, 32)
    value = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    byte = scales[:, :k // 32].astype(int)
    unit = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return (value * unit[..., None]).reshape(codes.shape[0], k)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def gelu_tanh(g):
    """g (1 + tanh w) / 2 as g / (1 + e^-2w): 1 + tanh w cancels for negative w
    (its relative error is 2^-53 / (1 + tanh w), e.g. 2^-24 at w = -10)."""
    w = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-2.0 * w))


def gated(gate, up, act):
    g = gate.astype(np.float64)
    return (act(g) * up.astype(np.float64)).astype(np.float32)


def norm(x, residual, rdtype, weight, eps):
    """(h as float32 values of rdtype, v fp32) of fp32 arrays."""
    h = rounded(x if residual is None else x + residual, rdtype)
    mean = (h.astype(np.float64) ** 2).sum(-1, keepdims=True) / h.shape[1]
    s = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
    v = h * s
    return h, v if weight is None else v * weight


def read_back(fmt, codes, scales, k):
    """Quantised rows as fp32 values: fmt "int4", "int8" or "mx4"."""
    if fmt == "mx4":
        return mx4_values(codes, scales, k).astype(np.float32)
    if fmt == "int4":
        b = codes.reshape(codes.shape[0], -1, 16)
        q = np.concatenate((b & 15, b >> 4), -1).astype(np.int8)
        q = np.where(q > 7, q - 16, q).reshape(codes.shape[0], k)
    else:
        q = codes
    return (q.reshape(q.shape[0], -1, 32).astype(np.float32) * scales[..., None]).reshape(q.shape[0], k)

"""What the quantised-row producers and the MXFP4 product are measured on.

Four operators, as a decoder layer uses them around its quantised products:

* ``norm``      residual addition + RMS norm, written as quantised rows (the
                input of q/k/v or gate/up), and the rows read back;
* ``glu``       gated activation, written as quantised rows (the input of the
                down projection), and the rows read back;
* ``quantise``  rows to MXFP4 (E2M1 codes, one power-of-two scale per 32),
                with or without the 32-point rotation, and read back;
* ``product``   y = a . w^T of two MXFP4 operands.

Quantised rows are returned as the values they stand for, in 16 bits: MXFP4
values are exact in bfloat16, int4 and int8 ones are rounded once to float16.

With ``own`` false, ``run`` computes the plain form in elementary torch
operations.  A code depends on every rounding before it, so the plain form
keeps the operators' definition step by step: row sums of squares and the
activation function in 64 bits, rounded once to 32, everything else one 32-bit
operation at a time.
"""
import functools
import math

import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-6
C32 = 0.1767766922712326  # 1/sqrt(32) rounded to 32 bits


def listed():
    return [
        # one generated token: the norm before q/k/v; the o projection's fp32 output joins the residual stream
        {"name": "norm 1x5120 mx4", "op": "norm", "rows": 1, "width": 5120, "format": "mx4_h32", "x": "float32", "residual": "float16", "pad": 0},
        # a speculative-verify block: int4 rows for the m <= 16 product
        {"name": "norm 16x5120 int4", "op": "norm", "rows": 16, "width": 5120, "format": "int4_small", "x": "float32", "residual": "float16", "pad": 0},
        # a prompt micro-batch: int8 rows for the exact int8 path
        {"name": "norm 512x5120 int8", "op": "norm", "rows": 512, "width": 5120, "format": "int8", "x": "float32", "residual": "bfloat16", "pad": 0},
        # a speculative-verify block between gate|up and down
        {"name": "glu 16x17408 mx4", "op": "glu", "rows": 16, "width": 17408, "format": "mx4_h32", "x": "float32", "act": "silu", "pad": 0},
        # the last, ragged micro-batch of a prompt, 16-bit gate and up in one packed matrix
        {"name": "glu 302x17408 int8", "op": "glu", "rows": 302, "width": 17408, "format": "int8", "x": "float16", "act": "gelu_tanh", "pad": 17408},
        # an expert layer's routed rows: 1024 tokens x top-8, gate|up packed
        {"name": "glu 8192x768 int4", "op": "glu", "rows": 8192, "width": 768, "format": "int4", "x": "float32", "act": "silu", "pad": 768},
        # a prompt micro-batch's activations
        {"name": "quantise 512x5120", "op": "quantise", "rows": 512, "width": 5120, "x": "float16", "rotate": True, "pad": 0},
        # a weight matrix, once per model load
        {"name": "quantise 17408x5120", "op": "quantise", "rows": 17408, "width": 5120, "x": "float32", "rotate": True, "pad": 0},
        # one generated token: the key projection
        {"name": "product 1x1024x5120", "op": "product", "rows": 1, "cols": 1024, "width": 5120, "y": "float32"},
        # a speculative-verify block: the gate projection
        {"name": "product 16x17408x5120", "op": "product", "rows": 16, "cols": 17408, "width": 5120, "y": "float32"},
        # a prompt's last micro-batch: the down projection
        {"name": "product 302x5120x17408", "op": "product", "rows": 302, "cols": 5120, "width": 17408, "y": "float32"},
        # a prompt micro-batch: gate|up packed, 16-bit outputs for the gated activation
        {"name": "product 512x34816x5120", "op": "product", "rows": 512, "cols": 34816, "width": 5120, "y": "float16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "glu", "quantise", "product", "product"])
    if op == "product":
        rows, cols, width = _log_uniform(rng, 1, 512), _log_uniform(rng, 1, 34816), 32 * _log_uniform(rng, 1, 544)
        while rows * cols * width > 512 * 34816 * 5120:
            cols = max(1, cols // 2)
        return {"op": op, "rows": rows, "cols": cols, "width": width, "y": rng.choice(list(TYPES))}
    rows, width = _log_uniform(rng, 1, 8192), 32 * _log_uniform(rng, 1, 544)
    while rows * width > 302 * 17408:
        rows = max(1, rows // 2)
    case = {"op": op, "rows": rows, "width": width, "x": rng.choice(list(TYPES)), "pad": rng.choice([0, 0, 1, 8, 96])}
    if op == "quantise":
        return {**case, "rotate": rng.random() < 0.7}
    formats = ["int4", "int8", "mx4", "mx4_h32"] + (["int4_small"] if rows <= 16 else [])
    case["format"] = rng.choice(formats)
    if op == "glu":
        return {**case, "act": rng.choice(["silu", "gelu_tanh"])}
    return {**case, "residual": rng.choice(["", "float16", "bfloat16", "float32"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, rows, width, dtype, pad=0):
    """N(0, 1) with 1 % of the channels 20 times as large (the same for every
    row), as a view of rows with `pad` more columns between them."""
    x = _normal(g, rows, width + pad)
    hot = torch.randperm(width, generator=g, device=DEV)[: (width + 50) // 100]
    x[:, hot] *= 20.0
    return x.to(dtype)[:, :width]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, rows, width = case["op"], case["rows"], case["width"]
    state = {"case": case}
    if op == "product":
        state["cols"] = case["cols"]
        state["a_codes"], state["a_scales"] = _mx4_rows(_normal(g, rows, width))
        state["w_codes"], state["w_scales"] = _mx4_rows(_normal(g, case["cols"], width) * 0.02)
        if own:  # the weights laid out once, and buffers that a serving loop keeps
            from hadamard_rotated_w4a4_amd import ops
            state["packed"] = ops.repack_mx4(state["w_codes"], state["w_scales"], case["cols"], width)
            state["y"] = torch.empty((rows, case["cols"]), dtype=TYPES[case["y"]], device=DEV)
            need = ops.gemm_mx4_workspace_bytes(rows, case["cols"], width)
            state["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
        return state
    dtype = TYPES[case["x"]]
    state["x"] = _activations(g, rows, width, dtype, case["pad"])
    if op == "norm":
        state["weight"] = 1.0 + 0.1 * _normal(g, width)
        state["residual"] = None
        if case["residual"]:
            state["residual"] = _activations(g, rows, width, TYPES[case["residual"]], case["pad"])
    if op == "glu":
        state["up"] = _normal(g, rows, width + case["pad"]).to(dtype)[:, :width]
        if case["pad"] == width:  # one packed product made both
            both = torch.cat((state["x"], state["up"]), 1)
            state["x"], state["up"] = both[:, :width], both[:, width:]
    return state


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _stage(v, h):
    """One butterfly stage over the last axis of 32: pairs (i, i + h)."""
    p = v.reshape(-1, 16 // h, 2, h)
    a, b = p[:, :, 0], p[:, :, 1]
    return torch.stack((a + b, a - b), dim=2).reshape(v.shape)


def _blocks(v, rotate):
    """[rows, width] in 32 bits as [rows, width/32, 32], rotated (not normalised) or not."""
    b = v.reshape(v.shape[0], -1, 32)
    return functools.reduce(_stage, (1, 2, 4, 8, 16), b) if rotate else b


def _mx4_blocks(b):
    """(codes 0..15 of each element, E8M0 byte of each block)."""
    amax = b.abs().amax(-1, keepdim=True)
    _, exponent = torch.frexp(amax)
    e = torch.where(amax > 0, exponent - 3, torch.full_like(exponent, -127)).clamp(-127, 127)
    a = torch.ldexp(torch.ldexp(b.abs(), -(e // 2)), -(e - e // 2))
    index = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    return index + 8 * torch.signbit(b).to(torch.uint8), (e + 127).to(torch.uint8).squeeze(-1)


def _mx4_rows(x):
    """MXFP4 rows as they lie in memory: codes [rows, width/2], element 2j in
    byte j's low half; scale bytes in rows of whole groups of 8, the rest 127."""
    codes, scales = _mx4_blocks(_blocks(x, False))
    codes = codes.reshape(x.shape[0], -1, 2)
    padded = torch.full((x.shape[0], -(-scales.shape[1] // 8) * 8), 127, dtype=torch.uint8, device=x.device)
    padded[:, : scales.shape[1]] = scales
    return codes[..., 0] | codes[..., 1] << 4, padded


def _mx4_value(codes, scale_bytes):
    """32-bit values of codes [..., 32] with one scale byte per block."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    return torch.ldexp(grid[codes.int()], scale_bytes.int().unsqueeze(-1) - 127)


def _mx4_matrix(codes, scales):
    """MXFP4 rows in memory as a 32-bit matrix."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1, 32)
    return _mx4_value(c, scales[:, : c.shape[1]]).reshape(codes.shape[0], -1)


def _int_values(b, top, rotated):
    """Blocks rounded to whole steps of max/top (half away from zero), as values."""
    d = b.abs().amax(-1, keepdim=True)
    d = d / torch.full_like(d, float(top))
    live = d >= 1.1754943508222875e-38
    inverse = torch.where(live, torch.ones_like(d) / d, torch.zeros_like(d))
    v = b * inverse
    t = torch.trunc(v)
    q = torch.where((v - t).abs() >= 0.5, t + torch.where(v < 0, -1.0, 1.0), t).clamp(-top, top)
    s = torch.where(live, d * C32 if rotated else d, torch.zeros_like(d))
    return q * s


def _quantised_values(v, form):
    """The values that the quantised rows of v (32 bits) stand for, in 16 bits."""
    shape = v.shape
    if form.startswith("mx4"):
        b = _blocks(v, form == "mx4_h32")
        return _mx4_value(*_mx4_blocks(b * C32 if form == "mx4_h32" else b)).reshape(shape).to(torch.bfloat16)
    return _int_values(_blocks(v, True), 127 if form == "int8" else 7, True).reshape(shape).to(torch.float16)


def _plain(state):
    case = state["case"]
    if case["op"] == "product":
        a = _mx4_matrix(state["a_codes"], state["a_scales"])
        w = _mx4_matrix(state["w_codes"], state["w_scales"])
        return torch.mm(a, w.t()).to(TYPES[case["y"]])
    x = state["x"]
    if case["op"] == "quantise":
        return _quantised_values(x.float(), "mx4_h32" if case["rotate"] else "mx4")
    if case["op"] == "glu":
        g = x.double()
        z = g if case["act"] == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)
        return _quantised_values((g / (1.0 + torch.exp(-z)) * state["up"].double()).float(), case["format"])
    r = state["residual"]
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    mean = h.double().square().mean(-1, keepdim=True)
    rstd = (1.0 / torch.sqrt(mean + EPS)).float()
    values = _quantised_values(h.float() * rstd * state["weight"], case["format"])
    return values if r is None else (h, values)


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def _own(state):
    from hadamard_rotated_w4a4_amd import ops
    case = state["case"]
    width = case["width"]
    if case["op"] == "product":
        return ops.gemm_mx4(state["packed"], state["a_codes"], state["a_scales"], case["cols"], width, y=state["y"], workspace=state["workspace"])
    if case["op"] == "quantise":
        form = ops.ACT_MX4_H32 if case["rotate"] else ops.ACT_MX4
        codes, scales = ops.quantize_mx4(state["x"], rotate=case["rotate"])
        return ops.dequantize_act(codes, scales, width, form, dtype=torch.bfloat16)
    form = {"int4": ops.ACT_INT4, "int4_small": ops.ACT_INT4_SMALL, "int8": ops.ACT_INT8, "mx4": ops.ACT_MX4, "mx4_h32": ops.ACT_MX4_H32}[case["format"]]
    values = torch.bfloat16 if case["format"].startswith("mx4") else torch.float16
    if case["op"] == "glu":
        codes, scales = ops.glu_quantize(state["x"], state["up"], form, act=ops.GLU_SILU if case["act"] == "silu" else ops.GLU_GELU_TANH)
        return ops.dequantize_act(codes, scales, width, form, dtype=values)
    codes, scales, h = ops.rms_norm_quantize(state["x"], state["weight"], EPS, form, residual=state["residual"])
    out = ops.dequantize_act(codes, scales, width, form, dtype=values)
    return out if state["residual"] is None else (h, out)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _exact_grid(v, form):
    """Blocks of 64-bit v on their 4- or 8-bit grid, in 64 bits."""
    b = v.reshape(-1, 32)
    if form != "mx4":
        i = torch.arange(32, device=v.device)
        parity = sum(((i[:, None] & i[None, :]) >> s) & 1 for s in range(5)) % 2
        b = torch.mm(b, (1.0 - 2.0 * parity.double()) / math.sqrt(32.0))
    top = b.abs().amax(1, keepdim=True)
    if form.startswith("mx4"):
        unit = torch.exp2(torch.floor(torch.log2(top.clamp_min(1e-300))).clamp(-125, 129) - 2)
        a = b.abs() / unit
        step = torch.exp2(torch.floor(torch.log2(a.clamp_min(1.0))) - 1.0)
        q = (torch.round(a / step) * step).clamp_max(6.0) * unit
    else:
        unit = top / (127 if form == "int8" else 7)
        q = torch.floor(b.abs() / unit.clamp_min(1e-300) + 0.5) * unit
    return (torch.sign(b) * q).reshape(v.shape)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "product":
        half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV)

        def matrix(codes, scales):
            low, high = codes.long() % 16, codes.long() // 16
            e = torch.stack((low, high), 2).reshape(codes.shape[0], case["width"])
            value = half[e % 8] * 0.5 * (1 - 2 * (e // 8))
            unit = torch.exp2(scales[:, : case["width"] // 32].double() - 127.0)
            return value * unit.repeat_interleave(32, dim=1)

        a, out = matrix(state["a_codes"], state["a_scales"]), []
        for lo in range(0, case["cols"], 4096):
            out.append(torch.mm(a, matrix(state["w_codes"][lo:lo + 4096], state["w_scales"][lo:lo + 4096]).t().contiguous()))
        return torch.cat(out, 1)
    x = state["x"].double()
    if case["op"] == "quantise":
        return _exact_grid(x, "mx4_h32" if case["rotate"] else "mx4")
    if case["op"] == "glu":
        y = x * torch.sigmoid(x) if case["act"] == "silu" else 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
        return _exact_grid(y * state["up"].double(), case["format"])
    h = x if state["residual"] is None else x + state["residual"].double()
    held = x if state["residual"] is None else h.to(state["residual"].dtype).double()
    v = held / torch.sqrt((held * held).sum(1, keepdim=True) / case["width"] + EPS) * state["weight"].double()
    values = _exact_grid(v, case["format"])
    return values if state["residual"] is None else (h, values)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    rows, width = case["rows"], case["width"]
    n = rows * width
    if case["op"] == "product":
        cols = case["cols"]
        return {"bytes": (rows + cols) * width * 17 / 32 + rows * cols * TYPES[case["y"]].itemsize, "flops": 2 * n * cols}
    size = TYPES[case["x"]].itemsize
    form = case.get("format", "mx4")
    held = n * 17 / 32 if form.startswith("mx4") else n * (9 / 8 if form == "int8" else 5 / 8)
    out = held + 2 * n  # the quantised rows, and the values read back
    if case["op"] == "quantise":
        return {"bytes": n * size + out, "flops": n * (8 if case["rotate"] else 3)}
    if case["op"] == "glu":
        return {"bytes": 2 * n * size + out, "flops": n * 12}
    r = TYPES[case["residual"]].itemsize if case["residual"] else 0
    return {"bytes": n * size + 2 * n * r + 4 * width + out, "flops": n * 12}

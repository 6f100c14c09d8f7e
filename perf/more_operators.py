"""What the 8-bit key/value cache's operators are measured on.

Two operators, what a decoder layer does between its q/k/v products and its
output product:

* ``append``  the q, k and v rows of new tokens (column ranges of one packed
              product): RMS norm of every q and k head, rotary positions (on one
              axis or several), k and v written into a paged cache of 8-bit
              values, q returned in 16 bits; and the blocks that were written,
              read back;
* ``attend``  causal attention of new tokens over that cache: single tokens,
              blocks of a few, prompts, ragged batches, sliding windows.

The cache holds E4M3 codes, with one power of two for the keys and one for the
values of every block of 32 tokens and head.  Keys and values that are read back
are returned as the values they stand for, exact in bfloat16.

With ``own`` false, ``run`` computes the plain form in elementary torch
operations.  A code depends on every rounding before it, so ``append`` keeps
the definition step by step: a head's sum of squares in 64 bits, everything else
one 32-bit operation at a time.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-6
BLOCK = 32  # tokens of one scale


def listed():
    return [
        # one generated token right after a short prompt: the smallest call
        _attend("attend 1x1 of 300", 24, 4, 256, 64, "bfloat16", seqs=1, tokens=1, context=300),
        # one generated token at the end of a very long document
        _attend("attend 1x1 of 131072", 24, 4, 256, 256, "bfloat16", seqs=1, tokens=1, context=131072),
        # a decode step of a serving batch, sequences of many lengths
        _attend("attend 32x1 of 16384", 48, 8, 128, 64, "float16", seqs=32, tokens=1, context=16384),
        # a speculative-verify block
        _attend("attend 1x16 of 8192", 24, 4, 256, 64, "bfloat16", seqs=1, tokens=16, context=8192),
        # a prompt's first micro-batch
        _attend("attend 1x512 of 512", 24, 4, 256, 64, "float16", seqs=1, tokens=512, context=512),
        # a prompt's last, ragged micro-batch
        _attend("attend 1x302 of 1838", 48, 8, 128, 32, "bfloat16", seqs=1, tokens=302, context=1838),
        # several chats' first turns together, odd lengths, layers with a sliding window
        _attend("attend 8x509 window 256", 32, 8, 64, 32, "float16", seqs=8, tokens=509, context=1021, window=256),
        # a micro-batch in the middle of a long document: the largest call
        _attend("attend 1x512 of 32768", 24, 4, 256, 128, "bfloat16", seqs=1, tokens=512, context=32768),
        # one generated token
        _append("append 1x1", 24, 4, 256, 64, "float32", "bfloat16", seqs=1, tokens=1, context=1000, rot=64),
        # a decode step of a serving batch
        _append("append 64x1", 48, 8, 128, 64, "bfloat16", "bfloat16", seqs=64, tokens=1, context=2048, rot=128, norm=False),
        # a prompt's micro-batch behind two others
        _append("append 1x512", 24, 4, 256, 64, "float32", "bfloat16", seqs=1, tokens=512, context=1536, rot=64),
        # prompts with images: positions in time, height and width
        _append("append 8x1023 three axes", 32, 4, 128, 32, "float16", "float16", seqs=8, tokens=1023, context=1500, rot=96, axes=3, interleaved=True),
    ]


def _attend(name, heads, kv_heads, dim, page, kind, *, seqs, tokens, context, window=0):
    return {"name": name, "op": "attend", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "type": kind,
            "seqs": seqs, "tokens": tokens, "context": context, "window": window}


def _append(name, heads, kv_heads, dim, page, kind, q_type, *, seqs, tokens, context, rot, axes=1, interleaved=False, norm=True):
    return {"name": name, "op": "append", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "type": kind, "q_type": q_type,
            "seqs": seqs, "tokens": tokens, "context": context, "rot": rot, "axes": axes, "interleaved": interleaved, "norm": norm}


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, kv_heads, dim = rng.choice([(24, 4, 256), (48, 8, 128), (32, 8, 64), (16, 2, 256), (28, 4, 128), (30, 2, 128), (16, 16, 64), (20, 1, 64)])
    case = {"heads": heads, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([32, 64, 96, 128, 256])}
    seqs = _log_uniform(rng, 1, 64)
    if rng.random() < 0.6:
        tokens = 1 if rng.random() < 0.5 else _log_uniform(rng, 2, 512)
        context = _log_uniform(rng, tokens, 131072)
        while seqs > 1 and (seqs * context * kv_heads * dim > 32 * 16384 * 1024 or seqs * tokens * context * heads * dim > 512 * 32768 * 6144):
            seqs = (seqs + 1) // 2
        while tokens * context * heads * dim > 512 * 32768 * 6144:
            context = max(tokens, context // 2)
        window = _log_uniform(rng, 1, 4096) if rng.random() < 0.25 else 0
        return {**case, "op": "attend", "type": rng.choice(["float16", "bfloat16"]), "seqs": seqs, "tokens": tokens, "context": context, "window": window}
    tokens = 1 if rng.random() < 0.4 else _log_uniform(rng, 2, 2048)
    while seqs > 1 and seqs * tokens * (heads + 2 * kv_heads) * dim > 8 * 1023 * 5120:
        seqs = (seqs + 1) // 2
    while tokens * (heads + 2 * kv_heads) * dim > 8 * 1023 * 5120:
        tokens = tokens // 2
    context = tokens + _log_uniform(rng, 1, 2048) - 1
    axes = rng.choice([1, 1, 3])
    return {**case, "op": "append", "type": rng.choice(list(TYPES)), "q_type": rng.choice(["float16", "bfloat16"]), "seqs": seqs, "tokens": tokens,
            "context": context, "rot": rng.choice([dim // 4, dim // 2, dim]), "axes": axes, "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.6}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _lengths(case):
    """(new tokens, total tokens) of each sequence: the first has the case's own,
    the others between a quarter of them and all."""
    out = []
    for b in range(case["seqs"]):
        part = 1.0 - 0.75 * ((b * 0.6180339887498949) % 1.0)
        n = max(1, round(case["tokens"] * part))
        out.append((n, max(n, round(case["context"] * part))))
    return out


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _hot(g, x, share=100):
    """x with 1 % of its last axis' channels 8 times as large."""
    width = x.shape[-1]
    x[..., torch.randperm(width, generator=g, device=DEV)[: (width + share // 2) // share]] *= 8.0
    return x


def _exponent(amax):
    """The smallest e, at least -127, with amax <= 448 * 2^e (-127 for 0)."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_min(-127)


def _random_blocks(g, blocks, heads, dim):
    """Codes and scale bytes of `blocks` x `heads` blocks of 32 tokens, as they lie in memory."""
    tokens = torch.exp(0.5 * _normal(g, blocks, 1, BLOCK, 1))
    k = _hot(g, _normal(g, blocks, heads, BLOCK, dim)) * tokens
    v = _normal(g, blocks, heads, BLOCK, dim) * tokens
    codes, scales = [], []
    for x, lay in ((k, _keys_as_stored), (v, _values_as_stored)):
        e = _exponent(x.abs().amax((-1, -2)))
        codes.append(lay(torch.ldexp(x, -e[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)))
        scales.append((e + 127).to(torch.uint8))
    return torch.stack(codes, 2), torch.stack(scales, 2)


def _keys_as_stored(c):
    """[..., 32 tokens, dim] -> [..., 32 * dim]: dims in chunks of 32, halves of
    16; a half holds every token's 16 bytes."""
    lead, dim = c.shape[:-2], c.shape[-1]
    return c.reshape(*lead, BLOCK, dim // 32, 2, 16).movedim(-4, -2).reshape(*lead, BLOCK * dim)


def _values_as_stored(c):
    """[..., 32 tokens, dim] -> [..., 32 * dim]: token 16i + 8q + 4h + r of
    channel 32c + d lies at 1024c + 512h + 16d + 8q + 4i + r."""
    lead, dim = c.shape[:-2], c.shape[-1]
    x = c.reshape(-1, 2, 2, 2, 4, dim // 32, 32)  # . i q h r c d
    return x.permute(0, 5, 3, 6, 2, 1, 4).reshape(*lead, BLOCK * dim)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lengths = _lengths(case)
    per_page = page // BLOCK
    need = [-(-total // page) for _, total in lengths]
    pool = sum(need) + 3
    codes, scales = _random_blocks(g, pool * per_page, kv_heads, dim)
    codes = codes.reshape(pool, per_page, kv_heads, 2, BLOCK * dim).movedim(2, 1).contiguous()
    scales = scales.reshape(pool, per_page, kv_heads, 2).movedim(2, 1).contiguous()
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [-1] * (max(need) - n))
        at += n
    starts = [0]
    for n, _ in lengths:
        starts.append(starts[-1] + n)
    ints = dict(dtype=torch.int32, device=DEV)
    state = {"case": case, "codes": codes, "scales": scales, "pages": torch.tensor(rows, **ints), "starts": torch.tensor(starts, **ints),
             "lens": torch.tensor([total for _, total in lengths], **ints), "total": starts[-1]}
    tokens = starts[-1]
    if case["op"] == "attend":
        state["q"] = _normal(g, tokens, heads, dim).to(TYPES[case["type"]])
        return state
    packed = _normal(g, tokens, (heads + 2 * kv_heads) * dim) * torch.exp(0.5 * _normal(g, tokens, 1))
    packed = _hot(g, packed).to(TYPES[case["type"]]).reshape(tokens, heads + 2 * kv_heads, dim)
    state["q"], state["k"], state["v"] = packed[:, :heads], packed[:, heads:heads + kv_heads], packed[:, heads + kv_heads:]
    state["q_weight"] = state["k_weight"] = None
    if case["norm"]:
        state["q_weight"], state["k_weight"] = 1.0 + 0.1 * _normal(g, dim), 1.0 + 0.1 * _normal(g, dim)
    # the table of a rotation's cosines and sines, one row a position
    half = case["rot"] // 2
    angles = torch.arange(case["context"] + 64, device=DEV, dtype=torch.float64)[:, None] * 1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    state["rope"] = torch.cat((torch.cos(angles), torch.sin(angles)), 1).float()
    state["positions"] = state["axes"] = None
    if case["axes"] > 1:
        state["positions"] = torch.randint(0, case["context"] + 64, (case["axes"], tokens), generator=g, **ints)
        state["axes"] = (torch.arange(half, device=DEV) * case["axes"] // half).to(torch.uint8)
    # the blocks that the new tokens reach, from their first slot on
    kept = [(total - n) % BLOCK for n, total in lengths]
    at = [0]
    for (n, _), before in zip(lengths, kept):
        at.append(at[-1] + n + before)
    state["read_starts"], state["read"] = torch.tensor(at, **ints), at[-1]
    state["slots"] = sum(-(-(n + before) // BLOCK) for (n, _), before in zip(lengths, kept))
    return state


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _stored_values(codes, scales, dim):
    """(keys, values) [..., 32 tokens, dim] in 32 bits of blocks as they lie in
    memory, [..., 2, 32 * dim]."""
    lead = codes.shape[:-2]
    x = torch.ldexp(codes.view(torch.float8_e4m3fn).float(), scales.int().unsqueeze(-1) - 127)
    k = x[..., 0, :].reshape(*lead, dim // 32, 2, BLOCK, 16).movedim(-2, -4).reshape(*lead, BLOCK, dim)
    v = x[..., 1, :].reshape(-1, dim // 32, 2, 32, 2, 2, 4).permute(0, 5, 4, 2, 6, 1, 3).reshape(*lead, BLOCK, dim)
    return k, v


def _plain_attend(state):
    case, q, pages = state["case"], state["q"], state["pages"].long()
    heads, kv_heads, dim, group = case["heads"], case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    seqs, longest = case["seqs"], case["tokens"]
    starts, lens = state["starts"].long(), state["lens"].long()
    count = starts[1:] - starts[:-1]
    # the sequences' keys and values, padded to one length: [seqs, kv_heads, length, dim]
    held = pages.clamp_min(0)
    k, v = _stored_values(state["codes"][held], state["scales"][held], dim)
    k = k.transpose(1, 2).reshape(seqs, kv_heads, -1, dim).transpose(2, 3).contiguous()
    v = v.transpose(1, 2).reshape(seqs, kv_heads, -1, dim)
    # and their new tokens' queries: [seqs, kv_heads, group * longest, dim]
    i = torch.arange(longest, device=DEV)
    row = (starts[:-1, None] + i).clamp_max(q.shape[0] - 1)
    rows = q[row].float().reshape(seqs, longest, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv_heads, group * longest, dim)
    scores = (torch.matmul(rows, k) / math.sqrt(dim)).reshape(seqs, kv_heads, group, longest, -1)
    j = torch.arange(scores.shape[-1], device=DEV)
    at = (lens - count)[:, None, None] + i[:, None]
    seen = (j <= at) & (j < lens[:, None, None])
    if case["window"]:
        seen = seen & (j > at - case["window"])
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1)
    out = torch.matmul(p.reshape(seqs, kv_heads, group * longest, -1), v).reshape(seqs, kv_heads, group, longest, dim)
    out = torch.where(total > 0, 1.0 / total, 0.0).unsqueeze(-1) * out
    seq = torch.repeat_interleave(torch.arange(seqs, device=DEV), count, output_size=state["total"])
    return out[seq, :, :, torch.arange(state["total"], device=DEV) - starts[seq]].reshape(-1, heads, dim).to(q.dtype)


def _rotated(x, weight, cos, sin, interleaved):
    """[tokens, heads, dim] in 32 bits: RMS norm where there is a weight, then the
    pairs of the leading channels rotated; cos and sin are [tokens, 1, pairs]."""
    if weight is not None:
        mean = x.double().square().mean(-1, keepdim=True)
        x = x * (1.0 / torch.sqrt(mean + EPS)).float() * weight
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _e4m3(x):
    """Values rounded to E4M3 (at most 448 in magnitude), ties to even, in 32 bits."""
    return x.to(torch.float8_e4m3fn).float()


def _plain_append(state):
    case = state["case"]
    dim, page, total = case["dim"], case["page"], state["total"]
    starts, lens, pages = state["starts"].long(), state["lens"].long(), state["pages"].long()
    seqs = torch.arange(case["seqs"], device=DEV)
    count = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(seqs, count, output_size=total)
    index = (lens - count)[seq] + torch.arange(total, device=DEV) - starts[seq]  # of each token in its sequence
    half = case["rot"] // 2
    if state["positions"] is None:
        cos, sin = state["rope"][index, :half], state["rope"][index, half:]
    else:
        at = state["positions"].long()[state["axes"].long()].t()
        pair = torch.arange(half, device=DEV)
        cos, sin = state["rope"][at, pair], state["rope"][at, half + pair]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    q = _rotated(state["q"].float(), state["q_weight"], cos, sin, case["interleaved"])
    k = _rotated(state["k"].float(), state["k_weight"], cos, sin, case["interleaved"])
    v = state["v"].float()
    # every block that a new token reaches: [slots, kv_heads, 32 tokens, dim]
    kept = (lens - count) % BLOCK
    blocks = (count + kept + BLOCK - 1) // BLOCK
    first = torch.cumsum(blocks, 0) - blocks
    slot_seq = torch.repeat_interleave(seqs, blocks, output_size=state["slots"])
    slot_block = (lens - count)[slot_seq] // BLOCK + torch.arange(state["slots"], device=DEV) - first[slot_seq]
    held = pages[slot_seq, slot_block * BLOCK // page]
    within = slot_block % (page // BLOCK)
    codes, scales = state["codes"][held, :, within], state["scales"][held, :, within]
    old = _stored_values(codes, scales, dim)
    old_index = slot_block[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)
    is_old = old_index < (lens - count)[slot_seq][:, None]
    place = first[seq] * BLOCK + kept[seq] + torch.arange(total, device=DEV) - starts[seq]
    read_seq = torch.repeat_interleave(seqs, count + kept, output_size=state["read"])
    read = first[read_seq] * BLOCK + torch.arange(state["read"], device=DEV) - state["read_starts"].long()[read_seq]
    out = []
    for x, before, byte in zip((k, v), old, (0, 1)):
        new = torch.zeros(state["slots"] * BLOCK, *x.shape[1:], device=DEV).index_copy(0, place, x)
        new = new.reshape(-1, BLOCK, *x.shape[1:]).transpose(1, 2)
        e = _exponent(new.abs().amax((-1, -2)))
        was = scales[..., byte].int() - 127
        e = torch.where(is_old.any(1, keepdim=True), torch.maximum(e, was), e)[..., None, None]
        both = torch.where(is_old[:, None, :, None], before, new)
        values = torch.ldexp(_e4m3(torch.ldexp(both, -e)), e).to(torch.bfloat16)
        out.append(values.transpose(1, 2).flatten(0, 1)[read])
    return q.to(TYPES[case["q_type"]]), out[0], out[1]


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def _own(state):
    from hadamard_rotated_w4a4_amd import ops
    case = state["case"]
    cache = state["codes"], state["scales"], state["pages"]
    if case["op"] == "attend":
        return ops.attention_kv(state["q"], *cache, state["starts"], state["lens"], window=case["window"])
    q = ops.append_kv(state["k"], state["v"], *cache, state["starts"], state["lens"], q=state["q"], rope=state["rope"], positions=state["positions"],
                      axes=state["axes"], interleaved=case["interleaved"], q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS,
                      dtype=TYPES[case["q_type"]])
    return q, *ops.read_kv(*cache, state["read_starts"], state["lens"], state["read"], dtype=torch.bfloat16)


def run(state):
    if own:
        return _own(state)
    return _plain_attend(state) if state["case"]["op"] == "attend" else _plain_append(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _exact_token(codes, scales, page_of, kind, token, dim):
    """[tokens, kv_heads, dim] in 64 bits of tokens (int64) of one sequence, byte by byte."""
    per_page = codes.shape[2]
    where, channel = page_of[token // (per_page * 32)], torch.arange(dim, device=DEV)
    block, t = token // 32 % per_page, (token % 32)[:, None]
    if kind == 0:
        byte = channel // 32 * 1024 + channel % 32 // 16 * 512 + t * 16 + channel % 16
    else:
        byte = channel // 32 * 1024 + t // 4 % 2 * 512 + channel % 32 * 16 + t // 8 % 2 * 8 + t // 16 * 4 + t % 4
    flat = codes.reshape(codes.shape[0], codes.shape[1], -1)
    offset = (block[:, None] * 2 + kind) * 32 * dim + byte
    c = flat[where[:, None], :, offset].transpose(1, 2).long()  # [tokens, kv_heads, dim]
    size, fraction = c // 8 % 16, (c % 8).double()
    value = torch.where(size > 0, (8 + fraction) * torch.exp2(size.double() - 10), fraction * 2.0 ** -9)
    unit = torch.exp2(scales[where, :, block, kind].double() - 127)
    return (1 - 2 * (c // 128)) * value * unit[..., None]


def _exact_grid(x, e):
    """x in 64 bits on the E4M3 grid of 2^e."""
    a = x.abs() / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp_max(448.0) * torch.exp2(e)


def _exact_rotated(x, weight, angle_table, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    c, s = angle_table
    half = c.shape[1]
    pair = torch.arange(half, device=DEV)
    one, two = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + half)
    out = x.clone()
    out[..., one] = x[..., one] * c[:, None] - x[..., two] * s[:, None]
    out[..., two] = x[..., two] * c[:, None] + x[..., one] * s[:, None]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    codes, scales, dim, group = state["codes"], state["scales"], case["dim"], case["heads"] // case["kv_heads"]
    results, begin = [], 0
    for b, (n, total) in enumerate(_lengths(case)):
        page_of = state["pages"][b].long()
        new = slice(begin, begin + n)
        begin += n
        if case["op"] == "attend":
            q = state["q"][new].double()
            low = max(0, total - n + 1 - case["window"]) if case["window"] else 0
            j = torch.arange(low, total, device=DEV)
            at = torch.arange(total - n, total, device=DEV)[:, None]
            hidden = (j > at) | ((j <= at - case["window"]) if case["window"] else (j < 0))
            k, v = _exact_token(codes, scales, page_of, 0, j, dim), _exact_token(codes, scales, page_of, 1, j, dim)
            out = torch.empty_like(q)
            for h in range(case["heads"]):
                score = torch.mm(q[:, h], k[:, h // group].t().contiguous()) * dim ** -0.5
                out[:, h] = torch.mm(torch.softmax(score.masked_fill(hidden, -math.inf), -1), v[:, h // group].contiguous())
            results.append((out,))
            continue
        first = total - n
        if state["positions"] is None:
            at = torch.arange(first, total, device=DEV)[:, None].expand(n, case["rot"] // 2)
        else:
            at = state["positions"][:, new].long().t()[:, state["axes"].long()]
        pair = torch.arange(case["rot"] // 2, device=DEV)
        turn = state["rope"][at, pair].double(), state["rope"][at, pair + case["rot"] // 2].double()
        q = _exact_rotated(state["q"][new], state["q_weight"], turn, case["interleaved"])
        sides = []
        for kind, x in ((0, _exact_rotated(state["k"][new], state["k_weight"], turn, case["interleaved"])), (1, state["v"][new].double())):
            kept = torch.arange(first // 32 * 32, first, device=DEV)
            pieces = []
            for lo in range(first // 32 * 32, total, 32):
                part = x[max(lo, first) - first:lo + 32 - first]
                e = torch.ceil(torch.log2(part.abs().amax((0, 2)) / 448.0)).clamp_min(-127.0)
                if lo < first:
                    e = torch.maximum(e, scales[page_of[lo // case["page"]], :, lo % case["page"] // 32, kind].double() - 127)
                    part = torch.cat((_exact_token(codes, scales, page_of, kind, kept, dim), part))
                pieces.append(_exact_grid(part, e[:, None]))
            sides.append(torch.cat(pieces))
        results.append((q, *sides))
    whole = tuple(torch.cat(parts) for parts in zip(*results))
    return whole[0] if case["op"] == "attend" else whole


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    heads, kv_heads, dim, lengths = case["heads"], case["kv_heads"], case["dim"], _lengths(case)
    tokens = sum(n for n, _ in lengths)
    if case["op"] == "attend":
        window = case["window"] or 1 << 40
        # tokens that some row sees, and pairs of a row and a token that it sees
        seen = sum(min(total, n - 1 + window) for n, total in lengths)
        pairs = sum(min(window, at + 1) for n, total in lengths for at in range(total - n, total))
        return {"bytes": seen * kv_heads * 2 * (dim + 1 / BLOCK) + 2 * tokens * heads * dim * TYPES[case["type"]].itemsize, "flops": 4 * pairs * heads * dim}
    kept = sum((total - n) % BLOCK for n, total in lengths)
    size = TYPES[case["type"]].itemsize
    inputs = tokens * (heads + 2 * kv_heads) * dim * size + tokens * min(case["rot"], dim) * 4
    # the codes written; the written blocks' codes read and their values in 16 bits
    cache = tokens * kv_heads * 2 * dim + (tokens + kept) * kv_heads * 2 * dim * 3
    return {"bytes": inputs + tokens * heads * dim * 2 + cache, "flops": tokens * (heads + 2 * kv_heads) * dim * 8}

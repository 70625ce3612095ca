"""What is measured of the serving operators next to the MuSe forward pass: rotary positions
with several axes, a key/value cache held in 4 bits (written and read back), and attention
over that cache.

Every case has a plain form (elementary torch operations in float32, angles in float64,
rounded once at the end) and, with ``own`` set, the calls a user makes of the library.

Rotary positions.  Pair i of P = sum(sections) channel pairs belongs to axis a(i) (the
sections in order) and turns by pos[b, a(i), n] * base^(-i/P); with a ladder for each axis
the exponent is -(i - first pair of the axis) / sections[a].  Pairs are channels (i, i + P),
or (2i, 2i + 1) when adjacent; channels from 2P on pass through.  The inverse turns back: it
is the gradient.

The cache.  uint8 [pages, Hkv, page / 32, 18 (D + Dv)]: tiles of 32 tokens, each holding the
codes of its keys (16 D bytes), of its values (16 Dv bytes), the key steps (bfloat16
[32, D / 32]) and the value steps (bfloat16 [32, Dv / 32]).  A group is 32 neighbouring
channels of one token and head: step = bfloat16(max|x| / 7), code = round_half_even(x / step)
in -7..7, held as code + 8 in four bits.  The order of the 32-bit words of a tile is that of
``_pack`` (a token's words are spread so that a warp's 16-byte loads are fragments of a matrix
instruction).  Token t of sequence b is at page page_table[b, t // page].

Attention over the cache.  Row m of sequence b (of M new rows) sees the tokens
t < lens[b] - M + m + 1; query head h reads key head h // (H / Hkv); a row that sees nothing
is zero, with -inf as its log-sum-exp.
"""
from __future__ import annotations

import math

import torch

own = False

INVERSE, ADJACENT, AXIS_LADDER = 1, 2, 4
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- cases

def listed():
    rope, kv, at = {"op": "rope"}, {"op": "cache"}, {"op": "attend"}
    return [
        # one new token of each of 16 sequences, queries and shared key heads, text positions
        dict(rope, name="rope_decode", B=16, H=16, Hk=4, N=1, D=128, dtype="bf16", sections="64",
             base=500000.0, flags=0, far=100000),
        # a video's queries and keys before the causal pass: time, height and width
        dict(rope, name="rope_video_n16k", B=4, H=8, Hk=8, N=16384, D=64, dtype="bf16",
             sections="8,12,12", base=10000.0, flags=0, far=2000),
        # gradients of an image's queries and keys in float32: two axes with a ladder each,
        # adjacent pairs, part of the channels, an odd length
        dict(rope, name="rope_grad_n5003_f32", B=2, H=16, Hk=16, N=5003, D=128, dtype="f32",
             sections="24,24", base=100.0, flags=INVERSE | ADJACENT | AXIS_LADDER, far=1024),
        # one new token of each sequence goes into the cache and comes back rounded
        dict(kv, name="cache_step", B=32, H=8, N=1, D=128, Dv=128, dtype="bf16", page=64, at=2047),
        # a prompt of the causal workload's length goes into the cache and comes back, as the
        # keys and values that later tokens will see
        dict(kv, name="cache_prompt_n16k", B=4, H=8, N=16384, D=64, Dv=64, dtype="bf16", page=256,
             at=0),
        # a float32 chunk of odd length behind a prefix that ends inside a tile
        dict(kv, name="cache_chunk_n1001_f32", B=3, H=4, N=1001, D=128, Dv=64, dtype="f32", page=32,
             at=77),
        # a long prompt of wide heads
        dict(kv, name="cache_prompt_n64k", B=1, H=16, N=65536, D=128, Dv=128, dtype="bf16",
             page=128, at=0),
        # the smallest step: one sequence, one token, a short cache
        dict(at, name="attend_short", B=1, H=8, Hkv=8, M=1, D=64, Dv=64, T=1021, ragged=False,
             dtype="bf16", page=64),
        # a serving batch with shared key heads and sequences of all lengths, one of them empty
        dict(at, name="attend_batch", B=48, H=32, Hkv=8, M=1, D=128, Dv=128, T=8192, ragged=True,
             dtype="bf16", page=64),
        # one long sequence at the width of the long-context workload
        dict(at, name="attend_n64k", B=2, H=16, Hkv=16, M=1, D=128, Dv=128, T=65536, ragged=False,
             dtype="bf16", page=256),
        # a chunk of drafted tokens checked at once, float32, several row tiles
        dict(at, name="attend_chunk_f32", B=3, H=16, Hkv=4, M=7, D=64, Dv=64, T=5000, ragged=True,
             dtype="f32", page=32),
        # the last chunk of a prompt against the cache
        dict(at, name="attend_chunk_m128", B=2, H=8, Hkv=2, M=128, D=128, Dv=128, T=16384,
             ragged=False, dtype="bf16", page=128),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    if op == "rope":
        axes = rng.choice([1, 2, 3, 4])
        P = D // 2 if rng.random() < 0.6 else rng.randrange(axes, D // 2 + 1)
        cuts = sorted(rng.sample(range(1, P), axes - 1))
        sections = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [P]))
        B, Hk = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 2, 4])
        N = _spread(rng, 1, max(1, min(65536, (60 << 20) // (B * (H + Hk) * D))))
        return dict(op=op, B=B, H=H, Hk=Hk, N=N, D=D, dtype=dtype, sections=sections,
                    base=rng.choice([100.0, 10000.0, 500000.0]), flags=rng.randrange(8),
                    far=rng.choice([100, 5000, 1000000]))
    Dv = D if rng.random() < 0.7 else 192 - D
    page = rng.choice([32, 64, 128, 256])
    if op == "cache":
        B, H = rng.choice([1, 2, 5, 16]), rng.choice([1, 2, 4, 8, 16])
        N = _spread(rng, 1, max(1, min(65536, (120 << 20) // (B * H * (D + Dv)))))
        return dict(op=op, B=B, H=H, N=N, D=D, Dv=Dv, dtype=dtype, page=page,
                    at=rng.choice([0, rng.randrange(500)]))
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 5, 8])
    M = rng.choice([1, 1, 1, 2, 5, 16, rng.randrange(1, 129)])
    # bounded by the largest listed case's cache and, for long chunks, by its products
    top = min(65536, int(250e6 / (Hkv * 256)), int(6e9 / (M * H * 256)))
    T = _spread(rng, 1, max(1, top))
    B = rng.choice([b for b in (1, 2, 3, 7, 16, 33) if b * T <= max(top, T)])
    return dict(op=op, B=B, H=H, Hkv=Hkv, M=M, D=D, Dv=Dv, T=T, ragged=rng.random() < 0.6,
                dtype=dtype, page=page)


def work(c):
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        x = c["B"] * (c["H"] + c["Hk"]) * c["N"]
        P = sum(int(s) for s in c["sections"].split(","))
        return {"bytes": 2 * x * c["D"] * es + 4 * c["B"] * c["N"] * len(c["sections"].split(",")),
                "flops": 6 * x * P}
    if c["op"] == "cache":
        x = c["B"] * c["H"] * c["N"] * (c["D"] + c["Dv"])
        # rows in, 4.5 bits a value out, the same in again, rows out
        return {"bytes": x * (2 * es + 2 * 9 / 16), "flops": 6 * x}
    lens = _lens_expected(c)
    rows = c["B"] * c["H"] * c["M"]
    return {"bytes": lens * c["Hkv"] * (c["D"] + c["Dv"]) * 9 / 16
            + rows * ((c["D"] + c["Dv"]) * es + 4),
            "flops": 2.0 * lens / c["B"] * rows * (c["D"] + c["Dv"])}


def _lens_expected(c):
    # a ragged batch's lengths are uniform over 0..T, with one sequence at T and one empty
    return c["B"] * c["T"] * (0.5 if c["ragged"] and c["B"] > 1 else 1.0)


# ------------------------------------------------------------------------- preparation

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    dt = DT[c["dtype"]]
    if c["op"] == "rope":
        s["sections"] = [int(x) for x in c["sections"].split(",")]
        A = len(s["sections"])
        s["Q"] = _randn(g, c["B"], c["H"], c["N"], c["D"]).to(dt)
        s["K"] = _randn(g, c["B"], c["Hk"], c["N"], c["D"]).to(dt)
        s["pos"] = _randint(g, 0, c["far"], c["B"], A, c["N"])
        return s
    if c["op"] == "cache":
        B, H, N, page = c["B"], c["H"], c["N"], c["page"]
        # keys with a few channels that are larger than the rest, as trained ones have
        gain = 1.0 + 7.0 * (torch.rand(c["D"], generator=g, device="cuda") < 0.05)
        s["K"] = (_randn(g, B, H, N, c["D"]) * gain).to(dt)
        s["V"] = _randn(g, B, H, N, c["Dv"]).to(dt)
        need = -(-(c["at"] + N) // page)
        order = torch.randperm(B * need, generator=g, device="cuda")
        s["page_table"] = order.reshape(B, need).to(torch.int32)
        s["start"] = torch.full((B,), c["at"], dtype=torch.int32, device="cuda")
        s["cache"] = torch.zeros(B * need, H, page // 32, 18 * (c["D"] + c["Dv"]), dtype=torch.uint8,
                                 device="cuda")
        return s
    B, H, Hkv, M, T, page = c["B"], c["H"], c["Hkv"], c["M"], c["T"], c["page"]
    need = -(-T // page)
    s["Q"] = _randn(g, B, H, M, c["D"]).to(dt)
    s["scale"] = c["D"] ** -0.5
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    if c["ragged"] and B > 1:
        lens[1:] = _randint(g, 0, T + 1, B - 1)
        lens[-1] = 0
    s["lens"] = lens
    s["page_table"] = torch.randperm(B * need, generator=g, device="cuda").reshape(B, need).to(torch.int32)
    cache = torch.empty(B * need, Hkv, page // 32, 18 * (c["D"] + c["Dv"]), dtype=torch.uint8,
                        device="cuda")
    n = max(1, (64 << 20) // (Hkv * page * (c["D"] + c["Dv"])))
    for p in range(0, B * need, n):  # pages at a time, to bound the temporaries
        m = min(n, B * need - p)
        K = _randn(g, m, Hkv, page, c["D"]).to(torch.bfloat16)
        V = _randn(g, m, Hkv, page, c["Dv"]).to(torch.bfloat16)
        cache[p:p + m] = _pack(*_quantise(K), *_quantise(V))
    s["cache"] = cache
    s["out"] = torch.empty(B, H, M, c["Dv"], dtype=dt, device="cuda")
    s["lse"] = torch.empty(B, H, M, dtype=torch.float32, device="cuda")
    if own:  # the workspace that a user's program keeps
        from clustered_softmax_attention_b200 import muse as m
        s["ws"] = m.workspace("muse_cache_attend", m.dims(s["Q"], s["out"], s["scale"]), Hkv)
    return s


# -------------------------------------------------------------------------- plain forms

def _rope_plain(X, pos, sections, base, flags):
    P, D, dev = sum(sections), X.shape[-1], X.device
    i = torch.arange(P, device=dev, dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=dev),
                                   torch.tensor(sections, device=dev), output_size=P)
    e = i / P
    if flags & AXIS_LADDER:
        width = torch.tensor(sections, device=dev, dtype=torch.float64)
        e = (i - (torch.cumsum(width, 0) - width)[axis]) / width[axis]
    angle = pos[:, axis].transpose(1, 2).double() * base ** -e  # [B, N, P]
    if flags & INVERSE:
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = X.float()
    if flags & ADJACENT:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
    else:
        a, b = x[..., :P], x[..., P:2 * P]
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], -1).flatten(-2) if flags & ADJACENT else torch.cat([u, v], -1)
    return torch.cat([y, x[..., 2 * P:]], -1).to(X.dtype)


def _quantise(X):
    """codes int32 [..., D] in -7..7 and steps bfloat16 [..., D / 32]."""
    x = X.float().unflatten(-1, (-1, 32))
    # quotients next to a half, and steps next to a rounding border, need more than 32 bits
    step = (x.abs().amax(-1, keepdim=True).double() / 7).float().to(torch.bfloat16)
    q = torch.where(step > 0, x.double() / step.double(), 0.0).round().clamp(-7, 7)
    return q.to(torch.int32).flatten(-2), step.squeeze(-1)


def _nibbles(u, order):
    """Words of eight codes (last axis, first code lowest) in the given order, as bytes."""
    shift = 4 * torch.arange(8, device=u.device, dtype=torch.int64)
    w = (u.long() << shift).sum(-1)
    w = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    return w.permute(order).flatten(3).contiguous().view(torch.uint8)


def _pack(kc, ks, vc, vs):
    """Codes and steps [pages, H, page, .] as tiles uint8 [pages, H, page / 32, 18 (D + Dv)]."""
    p, H, page, D = kc.shape
    Dv, T = vc.shape[-1], page // 32
    u = kc + 8
    if D == 128:  # token, quarter, group
        k = _nibbles(u.view(p, H, T, 32, 4, 4, 8), (0, 1, 2, 3, 5, 4))
    else:  # sixteen tokens: token % 8, quarter, token // 8, group
        k = _nibbles(u.view(p, H, T, 2, 2, 8, 2, 4, 8), (0, 1, 2, 3, 5, 7, 4, 6))
    u = vc + 8
    if Dv == 128:  # eight tokens: channel % 8, token pair, token % 2, half
        v = _nibbles(u.view(p, H, T, 4, 4, 2, 2, 8, 8).transpose(-1, -2), (0, 1, 2, 3, 7, 4, 5, 6))
    else:  # sixteen tokens: channel % 8, token pair, token // 8, token % 2
        v = _nibbles(u.view(p, H, T, 2, 2, 4, 2, 8, 8).transpose(-1, -2), (0, 1, 2, 3, 7, 5, 4, 6))
    steps = [x.view(p, H, T, -1).contiguous().view(torch.uint8) for x in (ks, vs)]
    return torch.cat([k, v] + steps, -1)


def _words(tiles, lo, hi):
    w = tiles[..., lo:hi].contiguous().view(torch.int32)
    shift = 4 * torch.arange(8, device=w.device, dtype=torch.int32)
    return (((w[..., None] >> shift) & 15) - 8).to(torch.int8)


def _codes(tiles, D):
    """Codes int8 and steps bfloat16 of the keys [n, H, page, .] and of the values, of tiles
    [n, H, page / 32, bytes]."""
    p, H, T, size = tiles.shape
    Dv = size // 18 - D
    k, v = _words(tiles, 0, 16 * D), _words(tiles, 16 * D, 16 * (D + Dv))
    if D == 128:
        k = k.view(p, H, T, 32, 4, 4, 8).permute(0, 1, 2, 3, 5, 4, 6)
    else:
        k = k.view(p, H, T, 2, 8, 4, 2, 2, 8).permute(0, 1, 2, 3, 6, 4, 7, 5, 8)
    if Dv == 128:
        v = v.view(p, H, T, 4, 8, 4, 2, 2, 8).permute(0, 1, 2, 3, 5, 6, 7, 8, 4)
    else:
        v = v.view(p, H, T, 2, 8, 4, 2, 2, 8).permute(0, 1, 2, 3, 6, 5, 7, 8, 4)
    at, out = 16 * (D + Dv), []
    for x, w in ((k, D), (v, Dv)):
        step = tiles[..., at:at + 2 * w].contiguous().view(torch.bfloat16)
        at += 2 * w
        out += [x.reshape(p, H, T * 32, w), step.view(p, H, T * 32, w // 32)]
    return out


def _values(code, step):
    return (code.unflatten(-1, (-1, 32)) * step.float()[..., None]).flatten(-2)


def _sequences(x, page_table):
    """Pages [n, H, page, D] as sequences [B, H, max_pages * page, D]."""
    y = x[page_table.long()]
    return y.transpose(1, 2).flatten(2, 3)


def _cache_plain(s):
    c = s["case"]
    N, at, page, D = c["N"], c["at"], c["page"], c["D"]
    table = s["page_table"].long()
    B, need = table.shape
    tiles = s["cache"]
    # whole pages: what is there already around the new tokens stays
    parts = []
    for new, was in zip((*_quantise(s["K"]), *_quantise(s["V"])), _codes(tiles, D)):
        full = _sequences(was, table).to(new.dtype)
        full[:, :, at:at + N] = new
        parts.append(full.unflatten(2, (need, page)).transpose(1, 2).flatten(0, 1).contiguous())
    tiles[table.flatten()] = _pack(*parts)
    kc, ks, vc, vs = (_sequences(x, table)[:, :, at:at + N] for x in _codes(tiles, D))
    return [_values(kc, ks).to(s["K"].dtype), _values(vc, vs).to(s["V"].dtype)]


def _attend_plain(s):
    c, Q = s["case"], s["Q"]
    B, H, M, D = Q.shape
    Hkv = c["Hkv"]
    kc, ks, vc, vs = (_sequences(x, s["page_table"])[:, :, :c["T"]] for x in _codes(s["cache"], D))
    K, V = _values(kc, ks), _values(vc, vs)
    q = Q.float().view(B, Hkv, H // Hkv * M, D)
    a = (q @ K.transpose(-1, -2) * s["scale"]).view(B, Hkv, H // Hkv, M, -1)
    t = torch.arange(K.shape[2], device=Q.device)
    m = torch.arange(M, device=Q.device)
    hide = t[None, None] >= (s["lens"][:, None] - M + m + 1)[..., None]
    a = a.masked_fill(hide[:, None, None], -torch.inf)
    top = a.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(a - top)
    z = p.sum(-1, keepdim=True)
    lse = (top + torch.log(z)).view(B, H, M)
    p = torch.where(z > 0, p / z, 0.0).view(B, Hkv, -1, p.shape[-1])
    return (p @ V).view(B, H, M, -1).to(Q.dtype), lse


def run(s):
    c = s["case"]
    if c["op"] == "rope":
        if own:
            from clustered_softmax_attention_b200 import muse as m
            return m.muse_rope_axes(s["Q"], s["pos"], s["sections"], c["base"], K=s["K"],
                                    flags=c["flags"])
        return [_rope_plain(x, s["pos"], s["sections"], c["base"], c["flags"])
                for x in (s["Q"], s["K"])]
    if c["op"] == "cache":
        if own:
            from clustered_softmax_attention_b200 import muse as m
            m.muse_cache_write(s["cache"], s["K"], s["V"], s["page_table"], s["start"])
            return m.muse_cache_read(s["cache"], s["page_table"], s["start"], c["N"], c["D"],
                                     dtype=s["K"].dtype)
        return _cache_plain(s)
    if own:
        from clustered_softmax_attention_b200 import muse as m
        return m.muse_cache_attend(s["Q"], s["cache"], s["page_table"], s["lens"], scale=s["scale"],
                                   out=s["out"], lse=s["lse"], ws=s["ws"])
    return _attend_plain(s)


# -------------------------------------------------------------- the definition, 64 bits

def _exact_rope(X, pos, sections, base, flags):
    P = sum(sections)
    Y = X.double().clone()
    first = 0
    for a, w in enumerate(sections):
        for j in range(w):
            i = first + j
            f = base ** (-j / w) if flags & AXIS_LADDER else base ** (-i / P)
            th = pos[:, a].double() * f * (-1.0 if flags & INVERSE else 1.0)
            lo, hi = (2 * i, 2 * i + 1) if flags & ADJACENT else (i, i + P)
            z = torch.complex(X[..., lo].double(), X[..., hi].double())
            z = z * torch.polar(torch.ones_like(th), th)[:, None]
            Y[..., lo], Y[..., hi] = z.real, z.imag
        first += w
    return Y


def _exact_round(X):
    """Every value as the cache holds it: its code times its group's step."""
    parts = []
    for g in X.double().split(32, -1):
        step = (g.abs().max(-1, keepdim=True).values / 7).float().bfloat16().double()
        code = torch.nan_to_num((g / step).round(), nan=0.0).clamp(-7, 7)
        parts.append(code * step)
    return torch.cat(parts, -1)


def _exact_values(tiles, D, lo, steps_at, keys):
    """Float64 [n, page, D] of one head's tiles uint8 [n, page / 32, bytes], by the place of
    each value's four bits."""
    dev = tiles.device
    n = tiles.shape[0]
    t = torch.arange(32, device=dev)[:, None]
    ch = torch.arange(D, device=dev)[None]
    if keys:
        q, w, nib = ch % 32 // 8, ch // 32, ch % 8
        word = t * 16 + q * 4 + w if D == 128 else \
            t // 16 * 128 + t % 8 * 16 + q * 4 + t // 8 % 2 * 2 + w
    else:
        r, nib = ch % 8, ch % 64 // 8
        word = t // 8 * 128 + r * 16 + t % 8 // 2 * 4 + t % 2 * 2 + ch // 64 if D == 128 else \
            t // 16 * 128 + r * 16 + t % 8 // 2 * 4 + t // 8 % 2 * 2 + t % 2
    byte = (lo + word * 4 + nib // 2).flatten()
    code = (tiles[:, :, byte].int() >> (nib % 2 * 4).expand(32, D).flatten()) % 16 - 8
    at = (steps_at + 2 * (t * (D // 32) + ch // 32)).flatten()
    bits = tiles[:, :, at].int() | tiles[:, :, at + 1].int() << 8
    step = (bits << 16).view(torch.float32).double()
    return (code.double() * step).view(n, -1, D)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return [_exact_rope(x, s["pos"], s["sections"], c["base"], c["flags"])
                for x in (s["Q"], s["K"])]
    if c["op"] == "cache":
        return [_exact_round(x) for x in (s["K"], s["V"])]
    Q, lens, table, tiles = s["Q"].double(), s["lens"].tolist(), s["page_table"].long(), s["cache"]
    B, H, M, D = Q.shape
    Dv, Hkv, page = c["Dv"], c["Hkv"], c["page"]
    out = torch.zeros(B, H, M, Dv, dtype=torch.float64, device=Q.device)
    lse = torch.full((B, H, M), -torch.inf, dtype=torch.float64, device=Q.device)
    G = H // Hkv
    for b in range(B):
        L = lens[b]
        pages = table[b, :-(-L // page)]
        see = torch.arange(M, device=Q.device) + (L - M + 1)
        live = see > 0
        if not bool(live.any()):
            continue
        for h in range(Hkv):
            one = tiles[pages, h]
            K = _exact_values(one, D, 0, 16 * (D + Dv), True)[..., :D].reshape(-1, D)[:L]
            V = _exact_values(one, Dv, 16 * D, 18 * D + 16 * Dv, False).reshape(-1, Dv)[:L]
            a = torch.einsum("gmd,td->gmt", Q[b, h * G:(h + 1) * G], K) * s["scale"]
            a = a.masked_fill(torch.arange(L, device=Q.device)[None] >= see[:, None], -torch.inf)
            z = torch.logsumexp(a, -1)
            o = torch.einsum("gmt,td->gmd", torch.exp(a - z.masked_fill(~live, 0.0)[..., None]), V)
            out[b, h * G:(h + 1) * G] = torch.where(live[:, None], o, 0.0)
            lse[b, h * G:(h + 1) * G] = torch.where(live, z, -torch.inf)
    return out, lse

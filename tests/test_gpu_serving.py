"""Rotary positions, the 4-bit cache and attention over it, against the float64 oracle.

Tolerances are worst-case bounds written beside each comparison: u = 2^-24 is half a float32
step, h = 2^-8 half a bfloat16 step (relative)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from clustered_softmax_attention_b200 import muse as m
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def randn(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def ok():
    assert m.muse_last_device_status() == 0


# ------------------------------------------------------------------- rotary positions

def rope_close(got, X, pos, sections, base, dtype, **kw):
    """The angle is off by at most u half turns (its rounding to float32) and sincospif by two
    steps (2^-22), the position's product with a float64 frequency by |pos| 2^-53; two products
    and a sum round three more times; the result once to its type."""
    ref = so.rope(X, pos, sections, base, **kw)
    size = np.abs(X).max(-1, keepdims=True) * 2
    far = np.abs(np.asarray(pos, dtype=np.float64)).max() * 2.0 ** -53
    tol = HALF[dtype] * np.abs(ref) + size * (np.pi * U + 2.0 ** -22 + 3 * U + far)
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) - tol)


ROPE = [  # B, H, Hk, N, D, sections, base, span of positions
    (1, 1, 0, 1, 64, (32,), 1e4, 1 << 31),
    (2, 3, 1, 37, 64, (8, 12, 12), 1e4, 2000),
    (3, 8, 2, 5, 128, (16, 24, 24), 5e5, 1 << 31),
    (1, 4, 4, 130, 128, (24, 24), 100.0, 1 << 20),
    (2, 2, 2, 33, 128, (1, 2, 3, 5), 1.0, 50),
    (1, 5, 0, 7, 64, (1,), 1e12, 1 << 31),
    (2, 9, 3, 64, 128, (13, 17), 1e4, 300),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("flags", range(8))
@pytest.mark.parametrize("B,H,Hk,N,D,sections,base,span", ROPE)
def test_rope_matches_oracle(B, H, Hk, N, D, sections, base, span, flags, dtype):
    rng = np.random.default_rng(flags)
    Q = randn(1, B, H, N, D, dtype=dtype)
    K = randn(2, B, Hk, N, D, dtype=dtype) if Hk else None
    pos = rng.integers(-span, span, (B, len(sections), N))
    kw = dict(inverse=bool(flags & 1), adjacent=bool(flags & 2), axis_ladder=bool(flags & 4))
    out = m.muse_rope_axes(Q, ints(pos), sections, base, K=K, flags=flags)
    for x, y in zip((Q, K), out if Hk else (out,)):
        rope_close(host(y), host(x), pos, sections, base, dtype, **kw)
        P = sum(sections)
        assert torch.equal(y[..., 2 * P:], x[..., 2 * P:])
    ok()


@pytest.mark.parametrize("adjacent", [0, m.MUSE_ROPE_ADJACENT])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rope_layouts_in_place_and_shared_positions(dtype, adjacent):
    """[B,N,H,D] memory in, shared positions, in place, a broadcast batch: the same values."""
    B, H, N, D, sec = 3, 4, 19, 64, (10, 6, 8)
    pos = ints(np.random.default_rng(0).integers(0, 99, (3, N)))
    X = randn(3, B, N, 3 * H, D, dtype=dtype)
    Q, K = X[:, :, :H].transpose(1, 2), X[:, :, H:2 * H].transpose(1, 2)
    ref_q, ref_k = m.muse_rope_axes(Q.contiguous(), pos.expand(B, 3, N).contiguous(), sec,
                                    K=K.contiguous(), flags=adjacent)
    kept = X.clone()
    a, b = m.muse_rope_axes(Q, pos, sec, K=K, flags=adjacent)
    assert torch.equal(a, ref_q) and torch.equal(b, ref_k) and torch.equal(X, kept)
    m.muse_rope_axes(Q, pos, sec, K=K, flags=adjacent, out=Q, k_out=K)
    assert torch.equal(Q, ref_q) and torch.equal(K, ref_k)
    assert torch.equal(X[:, :, 2 * H:], kept[:, :, 2 * H:])
    one = randn(4, 1, H, N, D, dtype=dtype)
    y = m.muse_rope_axes(one.expand(B, H, N, D), pos, sec, flags=adjacent)
    assert torch.equal(y, m.muse_rope_axes(one, pos, sec, flags=adjacent).expand(B, H, N, D))
    ok()


@pytest.mark.parametrize("sections,flags", [((32,), 0), ((9, 11), 2), ((8, 12, 12), 4)])
def test_rope_gradient_is_the_inverse(sections, flags):
    """sum(dO * R(X)) differentiated: against central differences of the oracle, and
    <R x, y> = <x, R^T y> on the GPU."""
    B, H, N, D = 1, 2, 5, 64
    rng = np.random.default_rng(7)
    pos = rng.integers(0, 50, (B, len(sections), N))
    X, dO = randn(5, B, H, N, D), randn(6, B, H, N, D)
    G = host(m.muse_rope_axes(dO, ints(pos), sections, 100.0, flags=flags | m.MUSE_ROPE_INVERSE))
    kw = dict(adjacent=bool(flags & 2), axis_ladder=bool(flags & 4))
    f = lambda x: (so.rope(x, pos, sections, 100.0, **kw) * host(dO)).sum()
    for idx in [(0, 0, 0, 0), (0, 1, 4, 17), (0, 0, 3, 33), (0, 1, 2, 63)]:
        d = np.zeros((B, H, N, D))
        d[idx] = 1e-4
        # R is linear: the difference is exact but for float64 rounding of sums of a few hundred
        # terms (1e-13 / 2e-4); the kernel as in rope_close
        np.testing.assert_allclose((f(host(X) + d) - f(host(X) - d)) / 2e-4, G[idx], atol=1e-5)
    rope_close(G, host(dO), pos, sections, 100.0, F32, inverse=True, **kw)


def test_rope_copies_infinities_and_nan_of_untouched_channels():
    X = randn(8, 1, 2, 9, 64, dtype=BF16)
    X[..., 40] = float("nan")
    X[..., 41] = float("inf")
    for flags in (0, m.MUSE_ROPE_ADJACENT):
        Y = m.muse_rope_axes(X, ints(np.arange(9)[None]), (20,), flags=flags)
        assert torch.equal(Y[..., 40:].view(torch.int16), X[..., 40:].view(torch.int16))
        assert torch.isfinite(Y[..., :40]).all()
    ok()


# ------------------------------------------------------------------------- the cache

class Store:
    """A cache with a shuffled page table, and what the oracle says it holds."""

    def __init__(self, B, Hkv, page, max_pages, D, Dv, seed=0, spare=2, fill=0):
        rng = np.random.default_rng(seed)
        n = B * max_pages + spare
        self.D, self.page = D, page
        self.cache = torch.full(m.muse_cache_shape(n, Hkv, page, D, Dv), fill, dtype=torch.uint8,
                                device="cuda")
        self.table_np = rng.permutation(n)[:B * max_pages].reshape(B, max_pages)
        self.table = ints(self.table_np)

    def values(self):
        """(K [B,Hkv,T,D], V [B,Hkv,T,Dv]) float64 from the bytes."""
        c = self.cache.cpu().numpy()
        n, Hkv, per, size = c.shape
        out = []
        for x in so.read_tiles(c.reshape(-1, size), self.D):
            x = x.reshape(n, Hkv, per * 32, -1)[self.table_np]          # [B, mp, Hkv, page, D]
            x = x.transpose(0, 2, 1, 3, 4)
            out.append(x.reshape(x.shape[0], Hkv, -1, x.shape[-1]))
        return out


def outliers(seed, *shape, dtype):
    """Rows with groups of very different sizes, ties and zeros."""
    x = randn(seed, *shape)
    x[..., 1::7] *= 30
    x[..., 32:64] *= 1e-3
    x[:, :, ::3, :32] = torch.round(x[:, :, ::3, :32] * 2) / 2     # many ties
    x[:, :, 1::5, 32:64] = 0
    x[:, :, 2::5, 32:64] *= 1e-38                                   # steps below the normal range
    x[:, :, 3::5, :32] *= 1e36
    return x.to(dtype)


WIDTHS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,Dv", WIDTHS)
@pytest.mark.parametrize("B,H,N,page,start", [
    (1, 1, 1, 32, [0]), (2, 3, 1, 64, [31, 32]), (2, 2, 33, 32, [0, 63]), (3, 1, 100, 128, [5, 0, 60]),
    (1, 4, 257, 256, [1]), (2, 2, 64, 1024, [0, 32])])
def test_write_then_read_holds_the_rounded_values(B, H, N, page, start, D, Dv, dtype):
    """The bytes hold exactly what the oracle says, tokens around them stay, and reading gives
    each value rounded once to its type."""
    mp = -(-(max(start) + N) // page) + 1
    s = Store(B, H, page, mp, D, Dv, seed=N, fill=0x5a)
    before = [x.copy() for x in s.values()]
    K, V = outliers(1, B, H, N, D, dtype=dtype), outliers(2, B, H, N, Dv, dtype=dtype)
    m.muse_cache_write(s.cache, K, V, s.table, ints(start))
    got = s.values()
    want = [so.held(host(K)), so.held(host(V))]
    for b in range(B):
        at = slice(start[b], start[b] + N)
        for g, w, o in zip(got, want, before):
            assert np.array_equal(g[b, :, at], w[b])
            assert np.array_equal(np.delete(g[b], np.r_[at], 1), np.delete(o[b], np.r_[at], 1),
                                  equal_nan=True)
    for t, w in zip(m.muse_cache_read(s.cache, s.table, ints(start), N, D, dtype=dtype), want):
        r = torch.tensor(w).to(F32).to(dtype)     # code * step is exact in float32
        assert torch.equal(t.cpu(), r)
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinities_and_nan_stay_in_their_group(dtype):
    s = Store(1, 1, 32, 2, 128, 64)
    K, V = randn(1, 1, 1, 40, 128, dtype=dtype), randn(2, 1, 1, 40, 64, dtype=dtype)
    K[0, 0, 3, 40], K[0, 0, 7, 100], V[0, 0, 9, 2] = float("nan"), float("-inf"), float("inf")
    m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
    k, v = m.muse_cache_read(s.cache, s.table, ints([0]), 40, 128, dtype=F32)
    for t, w in ((k, so.held(host(K))), (v, so.held(host(V)))):
        assert np.array_equal(host(t), w, equal_nan=True)
    assert int(torch.isnan(k).sum()) == 64 and int(torch.isnan(v).sum()) == 32
    ok()


def test_counts_strides_and_rows_left_as_they_were():
    """Ragged counts, [B,N,H,D] memory, a broadcast head; rows past a count neither written nor
    read."""
    B, H, N, D, page = 3, 2, 21, 64, 32
    s = Store(B, H, page, 3, D, D)
    empty = s.cache.clone()
    X = randn(3, B, N, H, 2 * D, dtype=BF16)
    K, V = X[..., :D].transpose(1, 2), X[..., D:].transpose(1, 2)
    counts, start = [0, 21, 9], [4, 40, 30]
    m.muse_cache_write(s.cache, K, V, s.table, ints(start), ints(counts))
    got = s.values()
    for g, x in zip(got, (K, V)):
        w = so.held(host(x))
        for b in range(B):
            assert np.array_equal(g[b, :, start[b]:start[b] + counts[b]], w[b, :, :counts[b]])
            rest = np.delete(g[b], np.r_[start[b]:start[b] + counts[b]], 1)
            assert (rest == 0).all()
    out = torch.full((2, B, N, H, D), 7.0, dtype=BF16, device="cuda")
    ko, vo = out[0].transpose(1, 2), out[1].transpose(1, 2)
    m.muse_cache_read(s.cache, s.table, ints(start), N, D, counts=ints(counts), out=(ko, vo))
    for t, x in ((ko, K), (vo, V)):
        w = torch.tensor(so.held(host(x))).to(BF16)
        for b in range(B):
            assert torch.equal(t[b, :, :counts[b]].cpu(), w[b, :, :counts[b]])
            assert (t[b, :, counts[b]:] == 7).all()
    ok()
    s.cache.copy_(empty)
    one = K[:, :1].expand(B, H, N, D)
    m.muse_cache_write(s.cache, one, one, s.table, ints([0] * B))
    assert np.array_equal(s.values()[1][:, :, :N], so.held(host(one)))


@pytest.mark.parametrize("what", ["page", "negative page", "past the table", "negative start",
                                  "far start", "count", "negative count"])
def test_bad_pages_and_positions_are_left_out_and_reported(what):
    B, H, N, D, page = 2, 1, 40, 64, 32
    s = Store(B, H, page, 3, D, D)
    K = randn(1, B, H, N, D, dtype=BF16)
    start, counts, good = [0, 10], None, np.ones((B, N), bool)
    tab = s.table_np.copy()
    if what == "page":
        tab[0, 1] = len(s.cache)
        good[0, 32:] = False
    elif what == "negative page":
        tab[0, 0] = -1
        good[0, :32] = False
    elif what == "past the table":
        start = [80, 10]
        good[0, 16:] = False
    elif what == "negative start":
        start = [-7, 10]
        good[0, :7] = False
    elif what == "far start":
        start = [2 ** 31 - 8, 10]
        good[0] = False
    else:
        counts = [41 if what == "count" else -1, 40]
        good[0] = what == "count"
    table, cnt = ints(tab), None if counts is None else ints(counts)
    m.muse_cache_write(s.cache, K, K, table, ints(start), cnt)
    assert m.muse_last_device_status() == 7
    want = so.held(host(K))
    for x in s.values():
        for b in range(B):
            for n in np.flatnonzero(good[b]):
                assert np.array_equal(x[b, :, start[b] + n], want[b, :, n])
    assert int((s.cache != 0).any(-1).sum()) > 0
    out = torch.full((2, B, H, N, D), 3.0, device="cuda")
    m.muse_cache_read(s.cache, table, ints(start), N, D, counts=cnt, out=(out[0], out[1]))
    assert m.muse_last_device_status() == 7
    for x in out:
        for b in range(B):
            assert np.array_equal(host(x[b])[:, good[b]], want[b][:, good[b]])
            assert (host(x[b])[:, ~good[b]] == 3).all()
    ok()


# -------------------------------------------------------------------- attention over it

def attend_close(got, lse, Q, s, lens, counts, scale, dtype):
    """A logit is a sum of 16-channel products and four scaled groups in float32: at most 20
    roundings (2u each where a matrix instruction cuts instead of rounding) of the partial sums,
    all below X = s sum|q k|, and a query of 22 bits; exp adds 2 steps of its result and the
    rounding of its argument.  So p is off by a factor of (1 + e), e = (42 u) X + 4 u and the
    normaliser by as much; p and then p * step are rounded to 11 bits (bfloat16 rows) or p * step
    to 22 (float32); their sums, over the tiles of a split, lose 2u a step of 16 tokens.

    A bfloat16 row's p and p * step are float16: below 2^-14 they are held to 2^-25, not to 11
    bits.  In their unit some step of the group is 2^-3 or more, and the normaliser 2^9 or more
    (the reference is some token's own logit, and weights there are 2^9): 2^-25 (1 + 2^3) 2^-9
    < 2^-30 of the group's largest step for each of T tokens, times a code of at most 7.  It shows
    only in channels where the tokens that the row attends are small or zero."""
    K, V = s.values()
    ref, ref_lse, A, X = so.cache_attend(host(Q), K, V, lens, counts, scale)
    least = np.zeros((Q.shape[0], Q.shape[1], 1, V.shape[-1]))
    if dtype == BF16:
        for b in range(Q.shape[0]):
            big = np.nan_to_num(np.abs(V[b][:, :lens[b]])).reshape(V.shape[1], lens[b], V.shape[-1] // 32, 32)
            big = big.max((1, 3), initial=0) / 7 * (1 + 2.0 ** -8) * lens[b] * 7 * 2.0 ** -30
            least[b, :, 0] = np.repeat(np.repeat(big, 32, -1), Q.shape[1] // V.shape[1], 0)
    T = max(lens)
    e = (42 * U * X + 4 * U)[..., None]
    p = 2.0 ** -10 if dtype == BF16 else 2.0 ** -21
    tol = HALF[dtype] * np.abs(ref) + A * (2 * e + p + 2 * U * (T / 16 + 40)) + least
    for b in range(Q.shape[0]):
        c = counts[b]
        d = np.abs(got[b, :, :c] - ref[b, :, :c])
        assert (d <= tol[b, :, :c]).all(), (b, float((d / (tol[b, :, :c] + 1e-300)).max()))
        r = ref_lse[b, :, :c]
        live = np.isfinite(r)
        assert np.array_equal(np.isneginf(lse[b, :, :c]), np.isneginf(r))
        t = (42 * U * X[b, :, :c] + 4 * U + 4 * U * np.abs(np.where(live, r, 0)) + 2 * U * (T / 16 + 40))
        assert (np.abs(lse[b, :, :c][live] - r[live]) <= t[live]).all()


def filled(B, Hkv, page, mp, D, Dv, T, dtype=BF16, seed=0, fill=0xff):
    s = Store(B, Hkv, page, mp, D, Dv, seed=seed, fill=fill)   # 0xff: NaN steps where unwritten
    if T:
        K, V = randn(seed + 1, B, Hkv, T, D), randn(seed + 2, B, Hkv, T, Dv)
        m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    return s


ATTEND = [  # B, H, Hkv, M, page, lens
    (1, 1, 1, 1, 32, [1]),
    (1, 8, 8, 1, 64, [33]),
    (4, 8, 2, 1, 64, [0, 1, 32, 200]),
    (2, 16, 1, 1, 128, [31, 129]),
    (3, 5, 1, 1, 32, [64, 65, 63]),
    (2, 4, 2, 3, 64, [2, 100]),          # a row that sees nothing
    (2, 10, 2, 7, 32, [300, 7]),
    (1, 40, 1, 1, 256, [500]),
    (2, 2, 1, 16, 64, [16, 90]),
    (1, 4, 2, 33, 64, [70]),
    (2, 8, 1, 128, 128, [128, 300]),
    (1, 3, 3, 65, 32, [40]),
    (1, 1, 1, 65, 64, [65]),             # more than 64 rows: blocks of 128
    (3, 8, 2, 20, 32, [0, 333, 130]),
    (2, 6, 3, 100, 128, [1000, 99]),
    (1, 1, 1, 1, 1024, [5000]),
    (40, 2, 2, 1, 32, [(37 * i) % 257 for i in range(40)]),
    (200, 1, 1, 1, 32, [(91 * i) % 1200 for i in range(200)]),   # more sequences than threads
    (2, 2, 2, 1, 64, [17000, 9000]),                             # long: stretches
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,Dv", WIDTHS)
@pytest.mark.parametrize("B,H,Hkv,M,page,lens", ATTEND)
def test_attend_matches_oracle(B, H, Hkv, M, page, lens, D, Dv, dtype):
    s = filled(B, Hkv, page, -(-max(lens) // page), D, Dv, max(lens))
    Q = randn(9, B, H, M, D, dtype=dtype)
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), scale=D ** -0.5)
    attend_close(host(out), host(lse), Q, s, lens, [M] * B, D ** -0.5, dtype)
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 4.0])
@pytest.mark.parametrize("M", [2, 20])
def test_attend_scales_and_sharp_softmax(M, scale, dtype):
    s = filled(2, 2, 64, 8, 64, 64, 450)
    Q = randn(3, 2, 8, M, 64, dtype=dtype)
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([450, 77]), scale=scale)
    attend_close(host(out), host(lse), Q, s, [450, 77], [M, M], scale, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [2, 40])
def test_attend_rows_of_very_different_sizes(M, dtype):
    """Queries and values from 1e-12 to 1e12, channels that are a thousand times the others', and
    values whose steps grow or fall along the sequence."""
    B, Hkv, T, D = 4, 1, 700, 64
    s = Store(B, Hkv, 64, 11, D, D)
    K, V = randn(1, B, Hkv, T, D), randn(2, B, Hkv, T, D)
    K[..., 5] *= 300
    ramp = 10.0 ** torch.linspace(-4, 4, T, device="cuda")[:, None]
    V[0] *= ramp
    V[1] *= ramp.flip(0)
    V[2] *= 1e-30
    V[3, ..., :32] *= 1e12
    m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    Q = randn(3, B, 4, M, D)
    Q[..., 5] *= 1e-2
    Q[:, 1] *= 1e-12
    Q[:, 2] *= 1e-3
    out, lse = m.muse_cache_attend(Q.to(dtype), s.cache, s.table, ints([T] * B), scale=0.3)
    attend_close(host(out), host(lse), Q.to(dtype), s, [T] * B, [M] * B, 0.3, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [1, 70])
def test_attend_a_large_value_that_the_softmax_ignores(M, dtype):
    """One token's values are 2^k times the others' and its logit far below: what the others
    give has to survive, whatever k."""
    D, T = 64, 110
    for k in (10, 20, 30, 60):
        s = Store(1, 1, 64, 2, D, D)
        K, V = randn(1, 1, 1, T, D) * 0.1, randn(2, 1, 1, T, D)
        Q = torch.ones(1, 1, M, D, device="cuda", dtype=dtype)
        K[0, 0, 33] = -400.0
        V[0, 0, 33] *= 2.0 ** k
        m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
        out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([T]), scale=1.0)
        attend_close(host(out), host(lse), Q, s, [T], [M], 1.0, dtype)


@pytest.mark.parametrize("M,H", [(1, 4), (6, 4), (40, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_counts_strides_and_rows_left_as_they_were(M, H, dtype):
    B, Hkv, D, Dv = 3, 2, 128, 64
    lens, counts = [90, 3, 41], [M, 0, max(1, M // 2)]
    s = filled(B, Hkv, 32, 3, D, Dv, 90)
    X = randn(4, B, M, H, D + 64, dtype=dtype)
    Q = X[..., :D].transpose(1, 2)
    out = torch.full((B, M, H, Dv), 5.0, dtype=dtype, device="cuda").transpose(1, 2)
    lse = torch.full((B, H, M), 5.0, device="cuda")
    ws = torch.full((m.muse_workspace_size("muse_cache_attend", m.dims(Q, out), Hkv),), 0xff,
                    dtype=torch.uint8, device="cuda")
    m.muse_cache_attend(Q, s.cache, s.table, ints(lens), ints(counts), 0.1, out, lse, ws)
    attend_close(host(out), host(lse), Q, s, lens, counts, 0.1, dtype)
    for b in range(B):
        assert (out[b, :, counts[b]:] == 5).all() and (lse[b, :, counts[b]:] == 5).all()
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,M", [(2, 5), (16, 5)])
def test_attend_nan_reaches_only_rows_and_groups_that_see_it(H, M, dtype):
    D, T = 64, 100
    s = Store(2, 1, 32, 4, D, 128, fill=0xff)
    K, V = randn(1, 2, 1, T, D), randn(2, 2, 1, T, 128)
    V[0, 0, 50, 70] = float("inf")       # group 2 of token 50
    K[1, 0, 97, 3] = float("nan")        # token 97: the last rows see it
    m.muse_cache_write(s.cache, K, V, s.table, ints([0, 0]))
    Q = randn(3, 2, H, M, D, dtype=dtype)
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([T, T]), scale=0.1)
    bad = torch.isnan(out)
    assert bad[0, :, :, 64:96].all() and not bad[0, :, :, :64].any() and not bad[0, :, :, 96:].any()
    assert not bad[1, :, :2].any() and bad[1, :, 2:].all()
    assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[1, :, :2]).all()
    assert torch.isnan(lse[1, :, 2:]).all()
    Q[0, 1, 2, 7] = float("nan")         # a query: its row alone
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([40, 40]), scale=0.1)
    bad = torch.isnan(out).all(-1)
    assert bad.sum() == 1 and bad[0, 1, 2] and torch.isnan(lse).sum() == 1
    ok()


@pytest.mark.parametrize("what", ["page", "long", "negative"])
@pytest.mark.parametrize("M,dtype", [(1, F32), (20, F32), (20, BF16), (70, BF16)])
def test_attend_bad_pages_and_lengths_are_left_out_and_reported(what, M, dtype):
    D = 64
    s = filled(2, 1, 32, 4, D, D, 128)
    tab, lens, seen = s.table_np.copy(), [100, 128], [np.arange(100), np.arange(128)]
    if what == "page":
        tab[0, 1] = 1 << 20
        seen[0] = np.delete(seen[0], np.r_[32:64])
    elif what == "long":
        lens[0], seen[0] = 1 << 30, np.arange(128)
    else:
        lens[0], seen[0] = -5, np.arange(0)
    Q = randn(3, 2, 2, M, D, dtype=dtype)
    out, lse = m.muse_cache_attend(Q, s.cache, ints(tab), ints(lens), scale=0.1)
    assert m.muse_last_device_status() == 7
    K, V = s.values()
    eff = [min(max(l, 0), 128) for l in lens]
    for b in range(2):
        for mm in (0, M - 1):
            see = seen[b][seen[b] < eff[b] - M + mm + 1]
            ref, rl, A, X = so.cache_attend(host(Q)[b:b + 1, :, mm:mm + 1], [K[b][:, see]],
                                            [V[b][:, see]], [len(see)], [1], 0.1)
            # weights of 11 bits twice and a result of 8 (bfloat16), values up to 5
            tol = 1e-5 if dtype == F32 else 5 * (2.0 ** -10 + 2.0 ** -8)
            assert np.allclose(host(out)[b:b + 1, :, mm:mm + 1], ref, atol=tol, rtol=0)
            assert np.allclose(host(lse)[b:b + 1, :, mm:mm + 1], rl, atol=1e-5)
    ok()


@pytest.mark.parametrize("M,pages", [(1, 32), (1, 400), (5, 400), (40, 32)])
def test_attend_repeats_exactly_and_does_not_depend_on_the_workspace(M, pages):
    """(a table of 400 pages has stretches instead of clusters)"""
    s = filled(3, 2, 64, pages, 64, 64, 2000)
    Q = randn(1, 3, 8, M, 64, dtype=BF16)
    lens = ints([2000, 17, 1234])
    n = m.muse_workspace_size("muse_cache_attend", m.dims(Q), 2)
    ref = None
    for fill in (0, 0xff, 0x7f):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out = m.muse_cache_attend(Q, s.cache, s.table, lens, scale=0.125, ws=ws)
        ref = ref or [x.clone() for x in out]
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("M", [1, 20])
def test_a_long_table_and_a_short_one_agree(M):
    """The same lengths in a table of their size and in one four hundred pages long: clusters and
    stretches of the same kernel, to float32 rounding of another split and the result's type."""
    lens = [1500, 0, 33, 999]
    s = filled(4, 2, 64, 400, 64, 128, 1500)
    for dtype in (F32, BF16):
        Q = randn(1, 4, 6, M, 64, dtype=dtype)
        a, la = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), scale=0.125)
        b, lb = m.muse_cache_attend(Q, s.cache, s.table[:, :24].contiguous(), ints(lens), scale=0.125)
        attend_close(host(a), host(la), Q, s, lens, [M] * 4, 0.125, dtype)
        attend_close(host(b), host(lb), Q, s, lens, [M] * 4, 0.125, dtype)
    ok()


def test_one_sequence_alone_and_in_a_batch():
    """A sequence's answer agrees with the same sequence answered alone, to float32 rounding of
    another split (A <= max|v| ~ 5: 1e-5 covers 2u (T / 16 + 40) A twice)."""
    s = filled(5, 1, 64, 20, 128, 128, 1200)
    Q = randn(1, 5, 8, 1, 128)
    lens = [1200, 900, 33, 0, 1]
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), scale=0.1)
    for b in range(5):
        o, l = m.muse_cache_attend(Q[b:b + 1], s.cache, s.table[b:b + 1], ints(lens[b:b + 1]), scale=0.1)
        assert torch.allclose(o[0], out[b], atol=2e-4, rtol=0) and torch.allclose(l[0], lse[b], atol=1e-5, rtol=0)


# ------------------------------------------------------------------ together, streams, graphs

def test_a_prompt_and_the_tokens_after_it():
    """As they are used: positions into Q and K, MuSe over the prompt, its keys and values into
    the cache, then tokens one by one; every answer is exact attention over what the cache
    holds."""
    B, H, N, D, block, page = 2, 4, 256, 64, 128, 64
    sec = (8, 12, 12)
    Q, K, V = (randn(i, B, H, N, D, dtype=BF16) * 0.3 for i in range(3))
    pos = ints(np.arange(N)[None, None].repeat(3, 1).repeat(B, 0))
    Qr, Kr = m.muse_rope_axes(Q, pos, sec, K=K)
    O = m.muse_causal_blocks(Qr, Kr, V, block, 16, 16, 3, scale=D ** -0.5)
    assert torch.isfinite(O).all()
    s = Store(B, H, page, N // page + 1, D, D)
    m.muse_cache_write(s.cache, Kr, V, s.table, ints([0] * B))
    # the cache's own prompt rows through MuSe: what later tokens see
    Kc, Vc = m.muse_cache_read(s.cache, s.table, ints([0] * B), N, D)
    assert torch.isfinite(m.muse_causal_blocks(Qr, Kc, Vc, block, 16, 16, 3, scale=D ** -0.5)).all()
    for t in range(3):
        q, k, v = (randn(10 + 3 * t + i, B, H, 1, D, dtype=BF16) * 0.3 for i in range(3))
        at = ints(np.full((B, 3, 1), N + t))
        q, k = m.muse_rope_axes(q, at, sec, K=k)
        m.muse_cache_write(s.cache, k, v, s.table, ints([N + t] * B))
        out, lse = m.muse_cache_attend(q, s.cache, s.table, ints([N + t + 1] * B), scale=D ** -0.5)
        attend_close(host(out), host(lse), q, s, [N + t + 1] * B, [1] * B, D ** -0.5, BF16)
    ok()


def test_replayed_steps_in_a_graph_follow_the_lengths():
    """A captured step (positions, write, attend) replayed with lengths, positions and rows
    updated in place; two graphs share one workspace."""
    B, H, Hkv, D, page = 3, 8, 2, 64, 32
    s = filled(B, Hkv, page, 8, D, D, 200, fill=0)
    q, k, v = (randn(i, B, h, 1, D, dtype=BF16) for i, h in ((1, H), (2, Hkv), (3, Hkv)))
    lens0 = np.array([199, 0, 63])
    pos, start, lens = ints(lens0[:, None, None]), ints(lens0), ints(lens0 + 1)
    out, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    ws = m.workspace("muse_cache_attend", m.dims(q), Hkv)

    def step():
        m.muse_rope_axes(q, pos, [32], K=k, out=qr, k_out=kr)
        m.muse_cache_write(s.cache, kr, v, s.table, start)
        m.muse_cache_attend(qr, s.cache, s.table, lens, scale=0.125, out=out, lse=lse, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for i in range(5):
        now = lens0 + i + 1
        pos.copy_(ints(now[:, None, None]))
        start.copy_(ints(now))
        lens.copy_(ints(now + 1))
        for j, x in enumerate((q, k, v)):
            x.copy_(randn(100 * i + j, *x.shape, dtype=BF16))
        graphs[i % 2].replay()
        attend_close(host(out), host(lse), qr, s, (now + 1).tolist(), [1] * B, 0.125, BF16)
    ok()


def test_calls_on_two_streams_at_once():
    s = filled(2, 2, 64, 32, 128, 128, 2000)
    Qs = [randn(i, 2, 16, 1, 128, dtype=BF16) for i in range(6)]
    lens = ints([2000, 1500])
    ref = [m.muse_cache_attend(q, s.cache, s.table, lens, scale=0.09)[0].clone() for q in Qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, q in enumerate(Qs * 4):
        with torch.cuda.stream(streams[i % 2]):
            got.append(m.muse_cache_attend(q, s.cache, s.table, lens, scale=0.09)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, ref[i % 6])
    ok()


def test_launch_counter_counts_the_serving_kernels():
    lib = m.lib()
    lib.muse_launch_counter.restype = m.ctypes.c_uint64
    s = filled(1, 1, 32, 2, 64, 64, 40)
    Q = randn(1, 1, 1, 1, 64)
    n0 = lib.muse_launch_counter()
    m.muse_rope_axes(Q, ints([[5]]), [32])
    m.muse_cache_read(s.cache, s.table, ints([0]), 40, 64)
    m.muse_cache_attend(Q, s.cache, s.table, ints([40]))
    assert lib.muse_launch_counter() - n0 >= 3


def test_a_replayed_chunk_of_many_rows_follows_the_lengths():
    """The form for many rows, captured: two graphs over one workspace, lengths and counts updated
    in place, a sequence with fewer rows than the others and one with none."""
    B, H, Hkv, M, D = 3, 8, 2, 40, 64
    s = filled(B, Hkv, 32, 20, D, D, 600)
    Q = randn(4, B, H, M, D, dtype=BF16)
    lens, counts = ints([600, 300, 40]), ints([M, 1, 0])
    out, lse = torch.zeros_like(Q), torch.zeros(B, H, M, device="cuda")
    ws = m.workspace("muse_cache_attend", m.dims(Q), Hkv)
    call = lambda: m.muse_cache_attend(Q, s.cache, s.table, lens, counts=counts, scale=0.125,
                                       out=out, lse=lse, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for i, (ln, cn) in enumerate((([599, 41, 40], [40, 1, 0]), ([7, 513, 1], [0, 40, 1]),
                                  ([128, 129, 600], [17, 33, 40]), ([600, 300, 40], [40, 1, 0]))):
        lens.copy_(ints(ln))
        counts.copy_(ints(cn))
        Q.copy_(randn(50 + i, *Q.shape, dtype=BF16))
        out.fill_(7.0)
        graphs[i % 2].replay()
        attend_close(host(out), host(lse), Q, s, ln, cn, 0.125, BF16)
        assert all((out[b, :, cn[b]:] == 7.0).all() for b in range(B))
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pages_past_four_gigabytes(dtype):
    """A cache of 15000 pages (4.4 GB), the sequence's pages at both ends of it: what is written,
    read and attended is what a small cache gives."""
    mp, Hkv, page, D = 3, 2, 1024, 128
    small = Store(1, Hkv, page, mp, D, D)
    big = torch.empty(m.muse_cache_shape(15000, Hkv, page, D, D), dtype=torch.uint8, device="cuda")
    assert big.numel() > 2 ** 32
    table = ints([[14999, 0, 14600]])
    T = mp * page - 5
    K, V = (randn(i, 1, Hkv, T, D, dtype=dtype) for i in (1, 2))
    got = []
    for cache, tab in ((small.cache, small.table), (big, table)):
        m.muse_cache_write(cache, K, V, tab, ints([0]))
        r = list(m.muse_cache_read(cache, tab, ints([0]), T, D, dtype=dtype))
        for H, M in ((4, 1), (8, 40)):
            r += m.muse_cache_attend(randn(3, 1, H, M, D, dtype=dtype), cache, tab, ints([T]), scale=0.1)
        got.append(r)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ok()


@pytest.mark.parametrize("M", [1, 40])
def test_sequences_that_share_pages(M):
    """A common beginning in the same pages, read by all."""
    s = filled(3, 2, 32, 12, 64, 64, 380)
    s.table_np[1:, :8] = s.table_np[0, :8]
    s.table = ints(s.table_np)
    lens = [380, 256, 300]
    Q = randn(5, 3, 8, M, 64, dtype=BF16)
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), scale=0.125)
    attend_close(host(out), host(lse), Q, s, lens, [M] * 3, 0.125, BF16)
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,M", [(2, 128), (16, 40), (64, 5)])
def test_a_padded_batch_of_one_long_chunk_and_single_tokens(H, M, dtype):
    """Several row blocks a head, of which most sequences use one."""
    B = 6
    s = filled(B, 2, 64, 10, 64, 64, 600)
    lens, counts = [600, 33, 1, 599, 0, 64], [M, 1, 1, 2, 1, 0]
    Q = randn(5, B, H, M, 64, dtype=dtype)
    out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), ints(counts), scale=0.125)
    attend_close(host(out), host(lse), Q, s, lens, counts, 0.125, dtype)
    assert all((out[b, :, counts[b]:] == 0).all() for b in range(B))
    ok()


FIRST_CALL = """
import torch
from clustered_softmax_attention_b200 import muse as m
H, M = {H}, {M}
cache = torch.zeros(m.muse_cache_shape(4, 2, 64, 64, 64), dtype=torch.uint8, device="cuda")
table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
K = torch.ones(1, 2, 200, 64, device="cuda", dtype=torch.bfloat16)
Q = torch.ones(1, H, M, 64, device="cuda", dtype=torch.bfloat16)
pos = torch.zeros(1, M, dtype=torch.int32, device="cuda")
zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 200, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    m.muse_cache_write(cache, K, K, table, zero)
    q = m.muse_rope_axes(Q, pos, [32])
    out, lse = m.muse_cache_attend(q, cache, table, lens, scale=0.125)
g.replay()
torch.cuda.synchronize()
want = float(torch.tensor(1 / 7, dtype=torch.bfloat16)) * 7
assert (out.float() - want).abs().max() <= want * (2 ** -8 + 2 ** -9), out
assert m.muse_last_device_status() == 0
print("replayed")
"""


@pytest.mark.parametrize("H,M", [(4, 1), (8, 40)])
def test_the_first_calls_of_a_process_are_captured(H, M):
    """What is looked up once a device is looked up during the capture.  Every value is code 7 of
    the step bf16(1/7) and the weights sum to one: off by the result's half step 2^-8 and weights
    of 11 bits, once for p and once for p step (2^-11 each), and float32 sums: below 2^-9."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(H=H, M=M)], capture_output=True, text=True,
                       timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "replayed" in r.stdout, r.stdout + r.stderr


def fine_close(got, Q, s, lens, counts, scale):
    """bfloat16 rows whose weights are not rounded to fewer bits than float32 arithmetic needs: as
    attend_close, but a weight is off by 2^-20 (two float16 pieces: the upper product's rounding is
    kept, the lower piece, at most 2^-10 of it, is rounded to 2^-21, and the weight's own lower piece to
    2^-22), or by 2^-23 in the unit where some step is 2^-3 and the normaliser 2^9: 2^-29 of the largest
    value.  Weights of 11 bits (2^-11, twice) would fail wherever a row's values cancel: a sum of T
    values of either sign is off by 2^-12 A / sqrt(T), more than all of this for short T."""
    K, V = s.values()
    ref, _, A, X = so.cache_attend(host(Q), K, V, lens, counts, scale)
    for b in range(Q.shape[0]):
        c, T = counts[b], lens[b]
        big = np.abs(V[b][:, :T]).max() * T * 2.0 ** -29
        e = (42 * U * X[b, :, :c] + 4 * U)[..., None]
        tol = HALF[BF16] * np.abs(ref[b, :, :c]) + A[b, :, :c] * (2 * e + 2.0 ** -20 + 2 * U * (T / 16 + 40)) + big
        d = np.abs(got[b, :, :c] - ref[b, :, :c])
        assert (d <= tol).all(), (b, int((d > tol).sum()), float((d / tol).max()))


FINE = [(8, 8, 1), (16, 2, 1), (16, 2, 2), (16, 2, 4), (16, 2, 8),   # 1, 8, 16, 32, 64 rows
        (4, 2, 40), (8, 2, 64)]                                        # 80, 256: the other form


@pytest.mark.parametrize("D,Dv", WIDTHS)
@pytest.mark.parametrize("H,Hkv,M", FINE)
def test_weights_of_bfloat16_rows_keep_their_bits(H, Hkv, M, D, Dv):
    lens = [32, 70, 200]
    s = filled(3, Hkv, 32, 8, D, Dv, 200)
    Q = randn(11, 3, H, M, D, dtype=BF16)
    out, _ = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), scale=0.02)
    fine_close(host(out), Q, s, lens, [M] * 3, 0.02)
    ok()


@pytest.mark.parametrize("D,Dv", [(64, 128), (128, 128)])
@pytest.mark.parametrize("H,M,counts", [(1, 66, [66, 65]), (4, 33, [17, 33]), (3, 128, [127, 23])])
def test_many_rows_in_warps_that_are_partly_filled(H, M, counts, D, Dv):
    """Two blocks of 64 value channels, rows that end inside a warp, items whole and split: lanes
    without a row take part in every load of the accumulators."""
    s = filled(2, 1, 64, 40, D, Dv, 2500)
    Q = randn(12, 2, H, M, D, dtype=BF16)
    for lens in ([2500, 1900], [200, 64]):
        out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints(lens), ints(counts), scale=0.1)
        attend_close(host(out), host(lse), Q, s, lens, counts, 0.1, BF16)
    ok()


@pytest.mark.parametrize("D,Dv", WIDTHS)
@pytest.mark.parametrize("what", ["nan", "inf", "zeros and a nan low", "zeros and a nan high", "tiny and a nan"])
@pytest.mark.parametrize("H,M", [(2, 4), (2, 40), (8, 16)])
def test_keys_that_are_all_nan_or_zero_but_for_one(H, M, what, D, Dv):
    """Sixteen neighbouring tokens whose only steps are NaN, zero or tiny: rows that see a NaN are NaN,
    and no others."""
    T, at = 256, 160
    s = Store(1, 1, 64, 4, D, Dv)
    K, V = randn(1, 1, 1, T, D), randn(2, 1, 1, T, Dv)
    first, last = at + 5, at + 5          # tokens that hold a NaN
    if what in ("nan", "inf"):
        K[0, 0, at:at + 16] = float(what)
        first, last = at, at + 15
    else:
        K[0, 0, at:at + 16] *= 1e-36 if "tiny" in what else 0
        K[0, 0, first, 40 if "high" in what else 3] = float("nan")
    m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
    Q = randn(3, 1, H, M, D, dtype=BF16)
    for length in (T, at + 8, at + 5 + M // 2, at):
        out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([length]), scale=0.1)
        sees = torch.arange(length - M, length).cuda() >= first
        assert torch.equal(torch.isnan(out).all(-1), sees.expand(1, H, M)), length
        assert torch.equal(torch.isnan(lse), sees.expand(1, H, M)) and torch.isfinite(out[:, :, ~sees]).all()
    ok()


def duration(f):
    """Shortest of some calls, ms."""
    f()
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("D,Dv", WIDTHS)
@pytest.mark.parametrize("H,M", [(16, 4), (32, 40)])
def test_values_that_begin_with_zeros(H, M, D, Dv):
    """Some groups zero over the first tokens, over all tokens, or over none: the answer, and about
    the time, of ordinary values (the next tile's size is what counts, not the first one's)."""
    B, Hkv, T = 2, 16, 2000
    s = Store(B, Hkv, 64, 32, D, Dv)
    K, V = randn(1, B, Hkv, T, D), randn(2, B, Hkv, T, Dv)
    Q = randn(3, B, H, M, D, dtype=BF16)
    call = lambda: m.muse_cache_attend(Q, s.cache, s.table, ints([T, T - 77]), scale=0.1)
    m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    plain = duration(call)
    V[0, :, :300] = 0
    V[1, :, :1100, :32] = 0
    V[1, ..., Dv - 32:] = 0
    m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    out, lse = call()
    attend_close(host(out), host(lse), Q, s, [T, T - 77], [M] * B, 0.1, BF16)
    assert (out[1, ..., Dv - 32:] == 0).all()
    # (recomputing a stretch on the CUDA cores took a hundred times as long)
    assert duration(call) < 5 * plain + 0.05
    ok()


@pytest.mark.parametrize("D,Dv", WIDTHS)
@pytest.mark.parametrize("H,M", [(4, 4), (4, 40), (2, 128)])
@pytest.mark.parametrize("odd", [[3], [0, 127, 128, 300], [200, 201, 260, 599], list(range(250, 290)) + [598]])
def test_a_few_values_of_another_size_count_by_their_weight(odd, H, M, D, Dv):
    """Tokens whose values are 2^40 times the others' and whose logits are so far below that both count,
    a few whose values are 2^-40 times, and a NaN: in the first tile of a stretch, at its end, behind
    what the earlier rows see.  Weights of 2^-40 of the largest count in full (float32 arithmetic: the
    bound of fine_close, its absolute term by the ordinary values)."""
    T = 600
    s = Store(1, 1, 32, 20, D, Dv)
    K, V = randn(1, 1, 1, T, D) * 0.2, randn(2, 1, 1, T, Dv)
    K[0, 0, odd] = -1.0
    V[0, 0, odd] *= 2.0 ** 40
    V[0, 0, 77:80] *= 2.0 ** -40
    m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
    Q = (torch.ones(1, H, M, D, device="cuda") + 0.1 * randn(3, 1, H, M, D)).to(BF16)
    scale = 28.0 / D                       # logits of the odd ones about -28: 2^-40
    out, _ = m.muse_cache_attend(Q, s.cache, s.table, ints([T]), scale=scale)
    Kh, Vh = s.values()
    ref, _, A, X = so.cache_attend(host(Q), Kh, Vh, [T], [M], scale)
    usual = np.delete(Vh[0][:, :T], odd, 1)
    e = (42 * U * X + 4 * U)[..., None]
    tol = HALF[BF16] * np.abs(ref) + A * (2 * e + 2.0 ** -20 + 2 * U * (T / 16 + 40)) \
        + np.abs(usual).max() * T * 2.0 ** -29
    d = np.abs(host(out) - ref)
    assert (d <= tol).all(), (int((d > tol).sum()), float((d / tol).max()))
    V[0, 0, T - 2, 40] = float("nan")
    m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
    bad = torch.isnan(m.muse_cache_attend(Q, s.cache, s.table, ints([T]), scale=scale)[0])
    sees = torch.arange(T - M, T).cuda() >= T - 2
    want = sees[:, None] & (torch.arange(Dv).cuda() // 32 == 1)
    assert torch.equal(bad, want.expand(1, H, M, Dv))
    ok()


@pytest.mark.parametrize("what", ["nan", "large", "growing"])
@pytest.mark.parametrize("M", [4, 40])
def test_values_of_another_size_cost_little(M, what):
    """One NaN or one large value of a long sequence takes about the time of ordinary values, and
    values that grow along the sequence a few times that (the stretch, or the rest of it, was
    recomputed: a hundred times)."""
    B, Hkv, T = 2, 2, 8192
    s = Store(B, Hkv, 64, 128, 128, 128)
    K, V = randn(1, B, Hkv, T, 128), randn(2, B, Hkv, T, 128)
    Q = randn(3, B, 8, M, 128, dtype=BF16)
    call = lambda: m.muse_cache_attend(Q, s.cache, s.table, ints([T, T]), scale=0.1)
    m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    plain = duration(call)
    if what == "growing":
        V *= 2.0 ** torch.linspace(-30, 30, T, device="cuda")[:, None]
    else:
        V[:, :, 5000, 7] = float("nan") if what == "nan" else 1e9
    m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    assert duration(call) < (16 if what == "growing" else 3) * plain + 0.05
    if what == "large":                  # where many stretches begin
        V[:, :, ::512, 7] = 1e9
        m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
        assert duration(call) < 4 * plain + 0.05
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 21, 2.0 ** 24, 2.0 ** 26, 2.0 ** 30])
@pytest.mark.parametrize("H,M", [(4, 1), (4, 16), (4, 40)])
def test_logits_far_from_zero(H, M, size, dtype):
    """Logits of either sign, of which float32 holds no fractions: the largest rounded ones share the
    row (attend_close: where X u is a step or more, any weights whose sum is one are right; what is not
    is a NaN, or a sum above the largest value)."""
    T = 300
    s = Store(2, 1, 32, 10, 64, 64)
    K, V = randn(1, 2, 1, T, 64), randn(2, 2, 1, T, 64)
    K[0] *= size
    K[1] = -size * (3 + 2.0 ** -8 * torch.arange(T, device="cuda")[:, None])
    m.muse_cache_write(s.cache, K, V, s.table, ints([0, 0]))
    Q = randn(3, 2, H, M, 64).abs().to(dtype)
    K, V = s.values()
    for length in (T, 129):
        out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([length] * 2), scale=0.25)
        ref, rl, A, X = so.cache_attend(host(Q), K, V, [length] * 2, [M] * 2, 0.25)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        # (42 u) X as in attend_close; log sums below log T
        assert (np.abs(host(lse) - rl) <= 42 * U * X + 4 * U * np.abs(rl) + 6).all()
        top = np.abs(V[:, :, :length]).max((1, 2))[:, None, None, :]
        assert (np.abs(host(out)) <= top * (1 + 2.0 ** -7)).all()
    ok()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,M", [(4, 4), (4, 40), (2, 128)])
@pytest.mark.parametrize("what", ["newest", "group", "tiny", "next to nothing"])
def test_keys_of_very_different_sizes_keep_their_logits(what, H, M, D):
    """The newest tokens' keys 2^30 times their neighbours', which earlier rows do not see; a group of
    channels 2^30 times the others where the queries are zero; a token's keys 2^-30 times the others',
    and all keys below 2^-126, with queries as far above: every row by what it sees (attend_close)."""
    T = 300
    s = Store(1, 1, 32, 10, D, 64)
    K, V = randn(1, 1, 1, T, D), randn(2, 1, 1, T, 64)
    Q = randn(3, 1, H, M, D)
    scale = 0.1
    if what == "newest":
        K[..., T - 2:, :] *= 2.0 ** 30
    elif what == "group":
        K[..., :32] *= 2.0 ** 30
        Q[..., :32] = 0
    elif what == "tiny":
        K[..., 200:203, :] *= 2.0 ** -30
        K[..., 100:117, 32:] *= 2.0 ** -60
    else:
        K *= 2.0 ** -127
        Q *= 2.0 ** 100
        scale = 2.0 ** 24
    m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
    Q = Q.to(BF16)
    for length in (T, T - 1, 256):
        out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([length]), scale=scale)
        attend_close(host(out), host(lse), Q, s, [length], [M], scale, BF16)
    ok()


@pytest.mark.parametrize("wait_limit_ns", [3_000_000, 0])
@pytest.mark.parametrize("T", [300, 4000])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_next_call_right(T, wait_limit_ns):
    """The many-row form with a part of its tiles withheld: every role winds down, the join finds no
    ends in the workspace that it can read by, and the next call is right.  (0: the default limit of 2 s,
    which all CTAs wait out together.)"""
    s = filled(2, 1, 32, 126, 64, 128, T)
    Q = randn(1, 2, 4, 40, 64, dtype=BF16)
    ws = torch.empty(m.muse_workspace_size("muse_cache_attend", m.dims(Q, randn(0, 2, 4, 40, 128, dtype=BF16)), 1),
                     dtype=torch.uint8, device="cuda")
    call = lambda: m.muse_cache_attend(Q, s.cache, s.table, ints([T, T // 2]), scale=0.1, ws=ws)
    ref = [x.clone() for x in call()]
    ok()
    m.muse_set_test_hooks(m.MUSE_TEST_WITHHOLD_CACHE, wait_limit_ns)
    try:
        ws.fill_(0xff)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        status = m.muse_last_device_status()
    finally:
        m.muse_set_test_hooks(0, 0)
    limit = (wait_limit_ns or 2_000_000_000) * 1e-6
    assert status == 6 and limit <= a.elapsed_time(b) < 2 * limit + 50
    assert all(torch.equal(x, y) for x, y in zip(call(), ref))
    ok()


def test_values_that_begin_with_zeros_take_the_straight_way_after_them():
    """64 rows a head, every item of one CTA beginning with four tiles of zeros: what follows takes the
    time of ordinary values (measured 1.04; in the unit of the zeros every tile took the wide way, 1.43)."""
    B, Hkv, T, D = 16, 28, 2048, 128
    s = Store(B, Hkv, 256, 8, D, D)
    K, V = (randn(i, 1, 1, T, D, dtype=BF16).expand(B, Hkv, T, D) for i in (1, 2))
    Q = randn(3, B, Hkv, 64, D, dtype=BF16)
    call = lambda: m.muse_cache_attend(Q, s.cache, s.table, ints([T] * B), scale=0.1)
    m.muse_cache_write(s.cache, K, V, s.table, ints([0] * B))
    plain = duration(call)
    V = V[:1, :1].clone()
    V[:, :, :128] = 0
    m.muse_cache_write(s.cache, K, V.expand(B, Hkv, T, D), s.table, ints([0] * B))
    assert duration(call) < 1.25 * plain
    ok()


@pytest.mark.parametrize("flags", [0, m.MUSE_ROPE_ADJACENT, m.MUSE_ROPE_INVERSE])
def test_rope_keeps_the_digits_of_a_small_sine(flags):
    """(1, 0) turned by every angle: its sine is off by a relative step or two (the function's, 2u each,
    and the result's rounding) and by an angle of 2^-31 half turns twice (the turn's 32 bits, the
    remainder of a rounded half turn), pi 2^-30, also where it is small; an angle rounded to float32 is
    off by pi 2^-25 there."""
    N, D, sec, base = 20000, 64, (1,), 1.0
    pos = np.arange(N)[None, None]
    X = torch.zeros(1, 1, N, D, device="cuda")
    X[..., 0] = 1
    y = host(m.muse_rope_axes(X, ints(pos), sec, base, flags=flags))[..., :2]
    ref = so.rope(host(X), pos, sec, base, inverse=bool(flags & 1), adjacent=bool(flags & 2))[..., :2]
    assert (np.abs(ref[..., 1]) < 2.0 ** -10).sum() > 5
    assert (np.abs(y - ref) <= 6 * U * np.abs(ref) + np.pi * 2.0 ** -30 + N * 2.0 ** -53).all()
    ok()


class Turned(torch.autograd.Function):
    """muse_rope_axes in a training graph."""

    @staticmethod
    def forward(ctx, Q, K, pos, flags):
        ctx.save_for_backward(pos)
        ctx.flags = flags
        return m.muse_rope_axes(Q, pos, (8, 12, 12), 100.0, K=K, flags=flags)

    @staticmethod
    def backward(ctx, dQ, dK):
        return (*m.muse_rope_axes(dQ.contiguous(), ctx.saved_tensors[0], (8, 12, 12), 100.0, K=dK.contiguous(),
                                  flags=ctx.flags ^ m.MUSE_ROPE_INVERSE), None, None)


@pytest.mark.parametrize("flags", [0, m.MUSE_ROPE_ADJACENT | m.MUSE_ROPE_AXIS_LADDER])
def test_rope_in_a_training_graph(flags):
    """Logits of turned queries and keys, keys shared by query heads: gradients against the same graph
    of float64 torch operations, in which a rotation is a product with its matrix.  A product's sums of
    64 and of N H terms in float32 are off by (64 + 2 N) u of their terms' sizes, a rotation as in
    rope_close (under 12 u); 256 u of the sizes that the gradients' terms reach."""
    B, H, Hk, N, D = 2, 4, 2, 9, 64
    Q, K = randn(1, B, H, N, D).requires_grad_(), randn(2, B, Hk, N, D).requires_grad_()
    pos = np.random.default_rng(0).integers(-50, 50, (B, 3, N))
    kw = dict(adjacent=bool(flags & 2), axis_ladder=bool(flags & 4))
    q, k = Turned.apply(Q, K, ints(pos), flags)
    assert q.requires_grad and not m.muse_rope_axes(Q, ints(pos), (8, 12, 12), flags=flags).requires_grad
    W = randn(3, B, H, N, N)
    ((q @ k.repeat_interleave(H // Hk, 1).transpose(-1, -2)) * W).sum().backward()
    eye = np.broadcast_to(np.eye(D)[None, :, None], (B, D, N, D))
    R = torch.tensor(so.rope(eye, pos, (8, 12, 12), 100.0, **kw)).permute(0, 2, 1, 3)  # [B, N, in, out]
    Q64, K64 = (x.detach().double().cpu().requires_grad_() for x in (Q, K))
    q64, k64 = (torch.einsum("bhnd,bnde->bhne", x, R) for x in (Q64, K64))
    ((q64 @ k64.repeat_interleave(H // Hk, 1).transpose(-1, -2)) * W.double().cpu()).sum().backward()
    for got, want, other in ((Q.grad, Q64.grad, K), (K.grad, K64.grad, Q)):
        size = 2 * float(W.abs().sum(-1).max()) * float(other.detach().abs().max()) * H
        assert (host(got) - want.numpy() <= 256 * U * size).all() and (want.numpy() - host(got) <= 256 * U * size).all()
    ok()


@pytest.mark.parametrize("H,M,dtype", [(16, 1, BF16), (16, 1, F32), (16, 8, BF16), (16, 40, BF16)])
def test_stretches_on_two_streams_at_once(H, M, dtype):
    """A table too long for clusters, and the form for many rows: partial sums and the join that reads
    them, on two streams with a workspace each, repeat what one stream gives."""
    s = filled(2, 2, 64, 400, 128, 128, 6000)
    Qs = [randn(i, 2, H, M, 128, dtype=dtype) for i in range(6)]
    lens = [ints([6000, 4500]), ints([77, 6000])]
    call = lambda q, i, ws: m.muse_cache_attend(q, s.cache, s.table, lens[i % 2], scale=0.09, ws=ws)
    wss = [m.workspace("muse_cache_attend", m.dims(Qs[0]), 2) for _ in range(2)]
    ref = [[x.clone() for x in call(q, i, wss[0])] for i, q in enumerate(Qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, q in enumerate(Qs * 4):
        k = (i // 2 + i) % 2
        with torch.cuda.stream(streams[k]):
            got.append(call(q, i, wss[k]))
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(pair, ref[i % 6])), i
    ok()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,M", [(4, 1), (4, 16), (4, 40)])
@pytest.mark.parametrize("qk", [(96, -96, 0), (98, 0, -112), (-100, 100, 0), (0, 0, -140)])
def test_the_ends_of_the_range(qk, H, M, dtype):
    """Keys, queries and the scale as far apart as float32 has them, values of 2^-60 and then of 2^46: as
    attend_close (scale times 2^-14 was held above 2^-123, which keys of 2^98 show)."""
    T, (k, q, c) = 300, qk
    s = Store(1, 1, 32, 10, 64, 64)
    K, V = randn(1, 1, 1, T, 64) * 2.0 ** k, randn(2, 1, 1, T, 64)
    V[:, :, :140] *= 2.0 ** -60
    V[:, :, 140:] *= 2.0 ** 46
    m.muse_cache_write(s.cache, K, V, s.table, ints([0]))
    Q = (randn(3, 1, H, M, 64) * 2.0 ** q).to(dtype)
    scale = 0.1 * 2.0 ** c
    for length in (T, 130):
        out, lse = m.muse_cache_attend(Q, s.cache, s.table, ints([length]), scale=scale)
        attend_close(host(out), host(lse), Q, s, [length], [M], scale, dtype)
    ok()

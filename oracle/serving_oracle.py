"""Float64 CPU oracle of the serving operators: rotary positions with several axes, the 4-bit
key/value cache, and causal attention over it.

TEST INFRASTRUCTURE ONLY, written from the definitions in include/muse.h; it shares no code
with the CUDA sources.  The pages that the library is built from describe the forward pass
only; these operators have no counterpart there.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------- rotary positions

def rope_frequencies(sections, base, axis_ladder=False):
    """(frequency, axis) of every pair."""
    P = sum(sections)
    f, axis, first = [], [], 0
    for a, w in enumerate(sections):
        for j in range(w):
            f.append(float(base) ** -(j / w if axis_ladder else (first + j) / P))
            axis.append(a)
        first += w
    return np.array(f), np.array(axis)


def rope(X, pos, sections, base, inverse=False, adjacent=False, axis_ladder=False):
    """X [B,H,N,D] turned by pos int [B,axes,N]; float64.  Far positions: the angle is reduced
    in extended precision before its sine and cosine are taken."""
    X = np.asarray(X, dtype=np.float64)
    f, axis = rope_frequencies(sections, base, axis_ladder)
    P = len(f)
    th = _reduce(np.asarray(pos)[:, axis], f)
    if inverse:
        th = -th
    c, s = (g(th).transpose(0, 2, 1)[:, None] for g in (np.cos, np.sin))
    i = np.arange(P)
    lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + P)
    Y = X.copy()
    Y[..., lo] = X[..., lo] * c - X[..., hi] * s
    Y[..., hi] = X[..., lo] * s + X[..., hi] * c
    return Y


def _reduce(pos, f):
    """pos * f modulo 2 pi, [B,P,N], with integers of any length: f as a fraction of a turn of 200
    bits."""
    two_pi = 62831853071795864769252867665590057683943387987502  # 2 pi * 10^49
    out = np.empty(pos.shape)
    for i in range(pos.shape[1]):
        num, den = float(f[i]).as_integer_ratio()
        turn = (num * 10 ** 49 << 200) // (den * two_pi)
        for b in range(pos.shape[0]):
            out[b, i] = [((int(p) * turn) % (1 << 200)) / (1 << 200) for p in pos[b, i]]
    return 2 * np.pi * out


# ------------------------------------------------------------------------- the 4-bit cache

def bf16(x):
    """The nearest bfloat16 (ties to even) of float64 values, as float64; values that float32
    holds, or quotients that are no nearer to a border than float32 can tell."""
    f = np.asarray(x, dtype=np.float64).astype(np.float32)
    bits = f.view(np.uint32).astype(np.uint64)
    up = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return np.where(np.isfinite(f), up.astype(np.uint32).view(np.float32), f).astype(np.float64)


def quantise(X):
    """(codes int [..., D], steps float64 [..., D/32]) of float64 rows [..., D]."""
    X = np.asarray(X, dtype=np.float64)
    g = X.reshape(*X.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        step = bf16(np.abs(g).max(-1) / 7.0)
    step = np.where(np.isfinite(g).all(-1), step, np.nan)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(step[..., None] > 0, g / step[..., None], 0.0)
    q = np.clip(np.rint(q), -7, 7)
    return q.reshape(X.shape).astype(np.int64), step


def held(X):
    """What the cache holds of rows X: code * step, float64."""
    q, step = quantise(X)
    return (q.reshape(*step.shape, 32) * step[..., None]).reshape(q.shape)


def tile_layout(D, Dv):
    """Where each value of a 32-token tile lies: (byte, shift) of the codes and the byte of the
    step, for keys [32, D] and for values [32, Dv]."""
    def place(word, nib, first):
        return first + 4 * word + nib // 2, 4 * (nib % 2)
    t = np.arange(32)[:, None]
    c = np.arange(D)[None]
    w, q, n = c // 32, c % 32 // 8, c % 8
    word = 16 * t + 4 * q + w if D == 128 else \
        128 * (t // 16) + 16 * (t % 8) + 4 * q + 2 * (t // 8 % 2) + w
    kb, ksh = place(word, n + 0 * t, 0)
    kst = 16 * (D + Dv) + 2 * (t * (D // 32) + c // 32)
    c = np.arange(Dv)[None]
    w, n, g = c // 64, c % 64 // 8, c % 8
    word = 128 * (t // 8) + 16 * g + 4 * (t % 8 // 2) + 2 * (t % 2) + w if Dv == 128 else \
        128 * (t // 16) + 16 * g + 4 * (t % 8 // 2) + 2 * (t // 8 % 2) + t % 2
    vb, vsh = place(word, n + 0 * t, 16 * D)
    vst = 18 * D + 16 * Dv + 2 * (t * (Dv // 32) + c // 32)
    return (kb, ksh, kst), (vb, vsh, vst)


def read_tiles(tiles, D):
    """(K [n,32,D], V [n,32,Dv]) float64 of tiles uint8 [n, bytes]."""
    n, size = tiles.shape
    out = []
    for b, sh, st in tile_layout(D, size // 18 - D):
        code = ((tiles[:, b].astype(np.int64) >> sh) & 15) - 8
        bits = tiles[:, st].astype(np.uint32) | tiles[:, st + 1].astype(np.uint32) << 8
        with np.errstate(invalid="ignore"):
            out.append(code * (bits << 16).view(np.float32).astype(np.float64))
    return out


# -------------------------------------------------------------------- attention over it

def cache_attend(Q, Ks, Vs, lens, counts, scale):
    """Causal attention of the newest counts[b] rows of Q [B,H,N,D] over what the cache holds:
    Ks[b] [Hkv,>=lens[b],D], Vs[b].  (O, lse, A, X): A = sum_t p_t |v_t| and X = the largest
    s sum_d |q_d k_td| a row sees, which error bounds are made of; rows past counts are NaN."""
    B, H, N, D = Q.shape
    Dv = Vs[0].shape[-1]
    O, A = np.full((B, H, N, Dv), np.nan), np.full((B, H, N, Dv), np.nan)
    lse, X = np.full((B, H, N), np.nan), np.full((B, H, N), np.nan)
    for b in range(B):
        G = H // Ks[b].shape[0]
        for h in range(H):
            k, v = Ks[b][h // G], Vs[b][h // G]
            for m in range(counts[b]):
                see = min(max(0, lens[b] - counts[b] + m + 1), lens[b])
                if see <= 0:
                    O[b, h, m], A[b, h, m], lse[b, h, m], X[b, h, m] = 0, 0, -np.inf, 0
                    continue
                q = np.asarray(Q[b, h, m], dtype=np.float64)
                x = scale * (k[:see] @ q)
                top = x.max()
                p = np.exp(x - top)
                z = p.sum()
                O[b, h, m] = p @ v[:see] / z
                A[b, h, m] = p @ np.abs(v[:see]) / z
                lse[b, h, m] = top + np.log(z)
                X[b, h, m] = (abs(scale) * (np.abs(k[:see]) @ np.abs(q))).max()
    return O, lse, A, X

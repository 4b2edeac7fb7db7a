"""Plain float64 references of the cache operators: rotary positions, the 8-bit K/V cache
(write, read, attention) and window attention with sinks.  Written from the formulas that
``include/clsa.h`` states, one loop per definition; no code of the library.
"""
from __future__ import annotations

import math

import numpy as np

# ------------------------------------------------------------------ rotary positions


def rope_freqs(rot, theta=10000.0, scaling="plain", factor=1.0, orig_len=1, beta_fast=32.0, beta_slow=1.0):
    """Radians a token of the rot / 2 pairs."""
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        turns = orig_len * f / (2 * math.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return g * f + (1 - g) * f / factor
    return f


def rope(x, pos, freqs, layout="half", mscale=1.0, inverse=False):
    """x [rows][heads][d], pos [n_pos]: row r has position pos[r % n_pos]."""
    x = np.asarray(x, dtype=np.float64)
    pairs = len(freqs)
    a = np.asarray(pos, dtype=np.float64)[np.arange(x.shape[0]) % len(pos), None] * freqs[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    if inverse:
        s = -s
    y = x.copy()
    for i in range(pairs):
        u, v = (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)
        y[..., u] = mscale * (x[..., u] * c[..., i] - x[..., v] * s[..., i])
        y[..., v] = mscale * (x[..., v] * c[..., i] + x[..., u] * s[..., i])
    return y


# ------------------------------------------------------------------ the 8-bit cache

E4M3_VALUES = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                        for e in range(16) for m in range(8)][:127])  # codes 0 .. 126; 127 is NaN


def e4m3_decode(codes):
    """Values of codes (uint8)."""
    codes = np.asarray(codes, dtype=np.int64)
    v = np.append(E4M3_VALUES, np.nan)[codes & 127]
    return np.where(codes & 128, -v, v)


def e4m3_encode(x):
    """Codes of values: the nearest, ties to the even code, beyond +-448 the last, NaN 127 (sign kept off)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3_VALUES, np.where(np.isnan(a), 0, a)), 0, 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3_VALUES[lo], E4M3_VALUES[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a >= 448.0, 126, code)
    code = code + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def kv8_scale(amax):
    """The smallest power of two in [2^-100, 2^119] with amax / s <= 448 (2^119 where none is)."""
    for e in range(-100, 120):
        if amax / 2.0 ** e <= 448.0:
            return 2.0 ** e
    return 2.0 ** 119


def kv8_write(codes, scales, X, start, count, block):
    """New codes [B][n][H][d] and scales [B][blocks][H] after rows X [B][T][H][d] were written."""
    codes, scales = codes.copy(), np.array(scales, dtype=np.float64)
    X = np.asarray(X, dtype=np.float64)
    B, T, H, _ = X.shape
    n = codes.shape[1]
    for b in range(B):
        c = min(max(int(count[b]), 0), T) if count is not None else T
        p0 = int(start[b])
        if c == 0 or p0 < 0 or p0 + c > n:
            continue
        for j in range(p0 // block, (p0 + c - 1) // block + 1):
            lo, hi = max(p0, j * block), min(p0 + c, (j + 1) * block)
            for h in range(H):
                x = X[b, lo - p0:hi - p0, h]
                fin = np.abs(x[np.isfinite(x)])
                s = kv8_scale(fin.max() if fin.size else 0.0)
                if lo > j * block:
                    old = scales[b, j, h]
                    s = max(s, old)
                    if s > old:
                        early = codes[b, j * block:lo, h]
                        codes[b, j * block:lo, h] = e4m3_encode(e4m3_decode(early) * (old / s))
                scales[b, j, h] = s
                codes[b, lo:hi, h] = e4m3_encode(x / s)
    return codes, scales


def kv8_values(codes, scales, block):
    """code * scale of a whole cache, [B][n][H][d]."""
    s = np.repeat(np.asarray(scales, dtype=np.float64), block, axis=1)[:, :codes.shape[1]]
    return e4m3_decode(codes) * s[..., None]


# ------------------------------------------------------------------ attention


def _rows(q, k, v, see, scale):
    """softmax of the seen scores, times v; (output, log-sum-exp), 0 and -inf where nothing is seen."""
    if not see.any():
        return np.zeros(v.shape[-1]), -math.inf
    s = (k[see] @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    return (p @ v[see]) / p.sum(), m + math.log(p.sum())


def attention(Q, K, V, tokens, scale=0.0):
    """Q [L][B][Hq][d] over K, V [B][n][Hkv][d] (or one sequence for all b): tokens[b] lists what b sees."""
    Q = np.asarray(Q, dtype=np.float64)
    L, B, Hq, d = Q.shape
    Hkv = K.shape[2]
    scale = scale if scale > 0 else 1 / math.sqrt(d)
    O, lse = np.zeros(Q.shape), np.full(Q.shape[:3], -math.inf)
    for b in range(B):
        kb, vb = K[b % K.shape[0]], V[b % V.shape[0]]
        tok = np.asarray(tokens[b], dtype=np.int64)
        all_of = np.ones(len(tok), dtype=bool)
        for l in range(L):
            for h in range(Hq):
                g = h // (Hq // Hkv)
                O[l, b, h], lse[l, b, h] = _rows(Q[l, b, h], kb[tok, g], vb[tok, g], all_of, scale)
    return O, lse


def window_sees(n, p, window, sinks):
    """Which of n tokens the row at position p sees."""
    j = np.arange(n)
    return (j <= p) & ((j > p - window) | (j < sinks))


def window_attention(Q, K, V, lens, window, sinks, scale=0.0):
    """Q [B][T][Hq][d]: row t of sequence b is the token lens[b] - T + t."""
    Q, K, V = (np.asarray(a, dtype=np.float64) for a in (Q, K, V))
    B, T, Hq, d = Q.shape
    Hkv = K.shape[2]
    scale = scale if scale > 0 else 1 / math.sqrt(d)
    O, lse = np.zeros(Q.shape), np.full(Q.shape[:3], -math.inf)
    for b in range(B):
        n = int(lens[b])
        for t in range(T):
            see = window_sees(n, n - T + t, window, sinks)
            for h in range(Hq):
                g = h // (Hq // Hkv)
                O[b, t, h], lse[b, t, h] = _rows(Q[b, t, h], K[b, :n, g], V[b, :n, g], see, scale)
    return O, lse

"""fp64 oracle of the calls that continue a sequence: rotary positions with either pairing and scaled
frequencies, the paged 8-bit cache (append, page copies) and attention over it.  Plain numpy, loops over
tokens and pages; shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

from .mmdit_oracle import positions


# ------------------------------------------------------------------ rotary

def frequencies(p: dict):
    """[(first channel, second channel, axis, frequency)] of every turned pair; p: theta, dims, half, scaling
    ("none", "linear", "ntk", "parts"), factors, trained, fast, slow."""
    out, at = [], 0
    for axis, d in enumerate(p["dims"]):
        f = p["factors"][axis]
        theta = p["theta"]
        if p["scaling"] == "ntk" and d > 2:
            theta *= f ** (d / (d - 2))
        for i in range(d // 2):
            w = theta ** (-2 * i / d)
            if p["scaling"] == "linear":
                w /= f
            elif p["scaling"] == "parts":
                turns = p["trained"][axis] * w / (2 * math.pi)
                g = min(max((turns - p["slow"]) / (p["fast"] - p["slow"]), 0.0), 1.0)
                w = g * w + (1 - g) * w / f
            pair = (at + i, at + i + d // 2) if p["half"] else (at + 2 * i, at + 2 * i + 1)
            out.append((*pair, axis, w))
        at += d
    return out


def rotary(x: np.ndarray, p: dict, layout, first, transpose: bool = False) -> np.ndarray:
    """x [B, N, H, D]; token n of item b has the position of the layout's token first[b] + n, (0, 0, 0) outside it."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    pos = positions(layout)
    sign = -1.0 if transpose else 1.0
    for b in range(x.shape[0]):
        for n in range(x.shape[1]):
            i = int(first[b]) + n
            at = pos[i] if 0 <= i < len(pos) else (0.0, 0.0, 0.0)
            for c1, c2, axis, w in frequencies(p):
                c, s = math.cos(at[axis] * w) * p["magnitude"], sign * math.sin(at[axis] * w) * p["magnitude"]
                y[b, n, :, c1] = x[b, n, :, c1] * c - x[b, n, :, c2] * s
                y[b, n, :, c2] = x[b, n, :, c1] * s + x[b, n, :, c2] * c
    return y


# ------------------------------------------------------------------ e4m3 and the cache

def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes, from sign, 4 exponent bits (bias 7) and 3 mantissa bits."""
    t = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[code] = math.nan if code & 127 == 127 else (-v if code & 128 else v)
    return t


E4M3 = e4m3_table()


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values, ties to the even mantissa, clipped to +-448; NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:127]  # ascending
    a = np.minimum(np.abs(np.nan_to_num(x)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    down, up = a - pos[lo], pos[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == pos[hi], hi, np.where(a == 0, 0, code))
    code = code + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def fit_scale(amax: float) -> float:
    """The power of two s with amax / s in (224, 448], 2^-60 at least."""
    s = 2.0 ** -60
    while amax / s > 448.0:
        s *= 2
    return s


def append(codes, scales, table, x, start, count, bad):
    """Stores x [B, N, H, D] (fp64; K already turned) into one half of the cache in place; codes uint8
    [P, H, T, D], scales [P, H], bad [B, N, H]: tokens whose codes become NaN (K), or None: values that are
    not finite become 0 (V)."""
    n_pages, heads, page, _ = codes.shape
    for b in range(x.shape[0]):
        n = min(max(int(count[b]), 0), x.shape[1])
        lo, hi = max(int(start[b]), 0), min(int(start[b]) + n, table.shape[1] * page)
        for j in range(lo // page, -(-hi // page) if hi > lo else 0):
            pid = int(table[b, j])
            if not 0 <= pid < n_pages:
                continue
            t0, t1 = max(lo, j * page), min(hi, (j + 1) * page)
            for h in range(heads):
                part = x[b, t0 - start[b]:t1 - start[b], h]
                fin = np.abs(part[np.isfinite(part)])
                s = fit_scale(fin.max() if fin.size else 0.0)
                old = float(scales[pid, h])
                if t0 > j * page:
                    if old > 0:
                        s = max(s, 2.0 ** math.ceil(math.log2(old)))
                    if s > old:
                        codes[pid, h, :t0 - j * page] = to_e4m3(E4M3[codes[pid, h, :t0 - j * page]] * (old / s))
                c = to_e4m3(np.where(np.isfinite(part), part, 0.0) / s)
                if bad is not None:
                    c[bad[b, t0 - start[b]:t1 - start[b], h]] = 127
                codes[pid, h, t0 - j * page:t1 - j * page] = c
                scales[pid, h] = s


def cache_attn(q, kc, vc, ks, vs, table, kv_len, q_len, causal: int, scale: float):
    """(o, lse, S, A): attention of q [B, N, H, D] over the cached tokens, per output the sum of p |v|, and per row
    the largest scaled sum of |q k| over the tokens it sees (the size of its scores' terms).  Rows behind q_len: NaN."""
    B, N, H, D = q.shape
    n_pages, Hk, page, _ = kc.shape
    o, S = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, A = np.full((B, H, N), np.nan), np.zeros((B, H, N))
    cap = table.shape[1] * page
    for b in range(B):
        kv, ql = min(max(int(kv_len[b]), 0), cap), min(max(int(q_len[b]), 0), N)
        ids = [int(table[b, n // page]) for n in range(kv)]
        there = np.array([0 <= i < n_pages for i in ids], bool)
        at = [(i, n % page) if 0 <= i < n_pages else (0, 0) for n, i in enumerate(ids)]
        for h in range(H):
            kh = h // (H // Hk)
            K = np.array([E4M3[kc[i, kh, s]] * float(ks[i, kh]) for i, s in at]).reshape(kv, D)
            V = np.array([E4M3[vc[i, kh, s]] * float(vs[i, kh]) for i, s in at]).reshape(kv, D)
            for n in range(ql):
                end = kv
                if causal:
                    p = kv - ql + n
                    end = 0 if p < 0 else min(kv, (p // causal + 1) * causal)
                see = np.nonzero(there[:end])[0]
                if not len(see):
                    o[b, n, h], S[b, n, h], lse[b, h, n] = 0.0, 0.0, -math.inf
                    continue
                s = (K[see] @ q[b, n, h]) * scale
                m = s.max()
                e = np.exp(s - m)
                w = e / e.sum()
                o[b, n, h], S[b, n, h] = w @ V[see], w @ np.abs(V[see])
                lse[b, h, n] = m + math.log(e.sum())
                A[b, h, n] = (np.abs(K[see]) @ np.abs(q[b, n, h])).max() * scale
    return o, lse, S, A

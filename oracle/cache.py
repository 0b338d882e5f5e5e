"""float64 oracle of rotary positions and of the bf16 / e4m3 paged cache (test
infrastructure only), in numpy, from the definitions in the library's header.
It never imports the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

D = 128
_CODES = None


def e4m3_values(codes) -> np.ndarray:
    """What e4m3 codes stand for: sign, four bits of exponent (bias 7), three of
    mantissa; no infinities, all ones NaN."""
    global _CODES
    if _CODES is None:
        c = np.arange(256)
        e, m = c >> 3 & 15, c & 7
        v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
        v[c & 127 == 127] = np.nan
        _CODES = np.where(c & 128, -v, v)
    return _CODES[np.asarray(codes, np.uint8)]


def rope(x, positions, inv_freq, interleaved: bool = False, scale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [rows, heads, 128] rotated, float64.  Positions times frequencies are
    products of 32 and 53 bits: longdouble keeps their fraction of a turn."""
    y = np.array(x, np.float64)
    f = np.asarray(inv_freq, np.longdouble)
    half = f.size
    t = np.asarray(positions, np.longdouble)[:, None] * f
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    t = (t - turn * np.rint(t / turn)).astype(np.float64)[:, None, :]
    cos, sin = scale * np.cos(t), scale * np.sin(t) * (-1 if inverse else 1)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = y[:, :, a], y[:, :, b]
    with np.errstate(invalid="ignore"):
        y[:, :, a], y[:, :, b] = u * cos - v * sin, v * cos + u * sin
    return y


def attention(q, k, v, block_table, seqlens_k, lq, scale: float | None = None):
    """q [total_q, h_q, 128] over k, v [num_pages, page, h_kv, 128], all values:
    (O float64 [total_q, h_q, 128], LSE float64 [h_q, total_q])."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    pages, page, h = k.shape[:3]
    h_q = q.shape[1]
    g = h_q // h
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, lse = np.zeros(q.shape), np.full((h_q, q.shape[0]), -np.inf)
    row = 0
    for r, (n, m) in enumerate(zip(seqlens_k, lq)):
        n, m = int(n), int(m)
        if 0 < n <= block_table.shape[1] * page:
            t = np.arange(n)
            pg = block_table[r, t // page].astype(np.int64)
            ok = (pg >= 0) & (pg < pages)
            pg = np.where(ok, pg, 0)
            kr, vr = (np.where(ok[:, None, None], x[pg, t % page], 0.0) for x in (k, v))
            here = slice(max(0, row), min(row + m, q.shape[0]))
            last = n - m + np.arange(m)[here.start - row:here.stop - row]
            seen = t[None, :] <= last[:, None]
            for a in range(h_q):
                with np.errstate(invalid="ignore", over="ignore"):
                    z = np.where(seen, scale * (q[here, a] @ kr[:, a // g].T), -np.inf)
                    any_key = seen.any(1)
                    top = np.where(any_key, z.max(1, initial=-np.inf), 0.0)
                    p = np.where(seen, np.exp(z - top[:, None]), 0.0)
                    total = p.sum(1)
                    vv = vr[:, a // g]
                    if np.isfinite(vv).all():
                        o = p @ vv
                    else:             # a value that a row does not attend is no term of its sum
                        o = np.stack([p[i, seen[i]] @ vv[seen[i]] for i in range(len(last))])
                    out[here, a] = np.where(any_key[:, None], o / np.where(any_key, total, 1.0)[:, None], 0.0)
                    lse[a, here] = np.where(any_key, top + np.log(np.where(any_key, total, 1.0)), -np.inf)
        row += m
    return out, lse

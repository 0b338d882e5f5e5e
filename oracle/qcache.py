"""float64 oracle of the serving operators (test infrastructure only): page
tables, the 4-bit K/V cache and attention over it, in numpy, from the
definitions in the library's header.  It never imports the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

D = 128


def chunk_bytes(group: int) -> int:
    return 2048 + 128 * (D // group)


def quantise(x: np.ndarray, group: int):
    """fp32-exact values [..., 128] -> codes uint8 [..., 128], f16 steps and minima
    [..., 128 / group].  The definition is in fp32, and so is this."""
    x = np.asarray(x, np.float32).reshape(*x.shape[:-1], D // group, group)
    bad = np.isnan(x).any(-1)
    with np.errstate(all="ignore"):
        x = np.clip(x, np.float32(-65504), np.float32(65504))
        low = np.where(bad, np.float16(np.nan), x.min(-1).astype(np.float16))
        lo32 = low.astype(np.float32)
        step = np.clip((x.max(-1) - lo32) / np.float32(15), np.float32(0), np.float32(65504)).astype(np.float16)
        step = np.where(bad, np.float16(0), step)
        s32 = step.astype(np.float32)
        inv = np.where(s32 > 0, np.float32(1) / s32, np.float32(0))
        code = np.clip(np.rint((x - lo32[..., None]) * inv[..., None]), 0, 15)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code.reshape(*code.shape[:-2], D), step, low


def values(code, step, low, group: int) -> np.ndarray:
    """step * code + minimum in float64."""
    c = code.reshape(*code.shape[:-1], D // group, group).astype(np.float64)
    return (c * step.astype(np.float64)[..., None] + low.astype(np.float64)[..., None]).reshape(code.shape)


def _places(t: int, group: int):
    """Byte and nibble of every K and V code of token t of a chunk, and the bytes of
    its f16 K steps, K minima, V steps, V minima."""
    n = D // group
    k, v = [], []
    for dim in range(D):
        q, j, i = dim // 32, dim % 32 // 8, dim % 8
        k.append((64 * t + 16 * j + 4 * q + i // 2, i % 2))
        y, r, i = dim // 32, dim % 32 // 4, dim % 4
        v.append((1024 + 512 * (t // 8) + 64 * r + 16 * (t % 8 // 2) + 8 * (t % 2) + 2 * y + i // 2, i % 2))
    ks = [2048 + 2 * (t * n + g) for g in range(n)]
    vs = [2048 + 64 * n + 2 * (((t % 8 // 2) * n + g) * 4 + (t // 8) * 2 + t % 2) for g in range(n)]
    return k, v, ks, [x + 32 * n for x in ks], vs, [x + 32 * n for x in vs]


def write(cache: np.ndarray, page: int, group: int, slots, k, v):
    """Quantise rows k, v [rows, h_kv, 128] into the cache (uint8 [pages, h_kv, page / 16, bytes]), in place."""
    slots, h, n = np.asarray(slots, np.int64), cache.shape[1], D // group
    parts = [quantise(k, group), quantise(v, group)]
    flat = cache.reshape(cache.shape[0], h, page // 16, -1)
    for t in range(16):
        rows = np.nonzero((slots % 16 == t) & (slots >= 0) & (slots < cache.shape[0] * page))[0]
        if not len(rows):
            continue
        at = (slots[rows] // page, slice(None), slots[rows] % page // 16)
        chunk = flat[at]                                         # [rows, h, bytes]
        kp, vp, ks, km, vs, vm = _places(t, group)
        for (code, step, low), places, sp, mp in zip(parts, (kp, vp), (ks, vs), (km, vm)):
            b = np.array([x for x, _ in places]).reshape(-1, 2)
            assert np.all(b[:, 0] == b[:, 1])                    # dims 2 i and 2 i + 1 share a byte
            c = code[rows]
            chunk[..., b[:, 0]] = c[..., 0::2] | (c[..., 1::2] << 4)
            for start, value in ((sp, step), (mp, low)):
                at16 = np.array([[x, x + 1] for x in start]).ravel()
                chunk[..., at16] = np.ascontiguousarray(value[rows]).view(np.uint8).reshape(len(rows), h, 2 * n)
        flat[at] = chunk


def read(cache: np.ndarray, page: int, group: int, slots):
    """(K, V) float64 [len(slots), h_kv, 128]: what the cache stands for; zeros where a slot is out of range."""
    h, n = cache.shape[1], D // group
    out = np.zeros((2, len(slots), h, D))
    slots = np.asarray(slots, np.int64)
    for t in range(16):
        rows = np.nonzero((slots % 16 == t) & (slots >= 0) & (slots < cache.shape[0] * page))[0]
        if not len(rows):
            continue
        chunk = cache[slots[rows] // page, :, slots[rows] % page // 16]        # [rows, h, bytes]
        kp, vp, ks, km, vs, vm = _places(t, group)
        for o, at, sp, mp in ((out[0], kp, ks, km), (out[1], vp, vs, vm)):
            b = np.array([x for x, _ in at])
            code = chunk[..., b] >> (4 * np.array([x for _, x in at], np.uint8)) & 15

            def halves(start):
                at16 = np.array([[x, x + 1] for x in start]).ravel()
                return np.ascontiguousarray(chunk[..., at16]).view(np.float16).reshape(len(rows), h, n)
            with np.errstate(invalid="ignore"):
                o[rows] = values(code, halves(sp), halves(mp), group)
    return out[0], out[1]


def attention(q, cache, page: int, group: int, block_table, seqlens_k, lq, scale: float | None = None):
    """q [total_q, h_q, 128] -> (O float64 [total_q, h_q, 128], LSE float64 [h_q, total_q])."""
    q = np.asarray(q, np.float64)
    h_q, h = q.shape[1], cache.shape[1]
    g = h_q // h
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, lse = np.zeros(q.shape), np.full((h_q, q.shape[0]), -np.inf)
    row = 0
    for r, (n, m) in enumerate(zip(seqlens_k, lq)):
        n, m = int(n), int(m)
        if 0 < n <= block_table.shape[1] * page:
            t = np.arange(n)
            pg = block_table[r, t // page].astype(np.int64)
            ok = (pg >= 0) & (pg < cache.shape[0])
            k, v = read(cache, page, group, np.where(ok, pg * page + t % page, -1))
            for i in range(m):
                last = n - m + i
                if last < 0:
                    continue
                for a in range(h_q):
                    z = scale * (k[:last + 1, a // g] @ q[row + i, a])
                    top = z.max()
                    p = np.exp(z - top)
                    out[row + i, a] = p @ v[:last + 1, a // g] / p.sum()
                    lse[a, row + i] = top + np.log(p.sum())
        row += m
    return out, lse


def page_tables(block_table, seqlens, new_lens, free_pages, head: int, page: int, num_pages: int, capacity: int):
    """(block_table, cu_seqlens_q, seqlens_k, positions, slots, free_next, any refused)."""
    table = block_table.copy()
    batch, width = table.shape
    cu, total = np.zeros(batch + 1, np.int64), np.array(seqlens, np.int64)
    positions, slots = np.zeros(capacity, np.int64), np.full(capacity, -1, np.int64)
    off = taken = 0
    avail = len(free_pages) - head if head >= 0 else 0
    refused = head < 0 or head > len(free_pages)
    for r in range(batch):
        old, new = int(seqlens[r]), int(new_lens[r])
        ok = old >= 0 and new >= 0 and old + new <= 2 ** 31 - 1 and -(-(old + new) // page) <= width
        need = -(-(old + new) // page) - -(-old // page) if ok else 0
        start = int(cu[r])
        cu[r + 1] = start + max(0, new)
        ok = ok and (need == 0 or off + need <= avail) and (new == 0 or start + new <= capacity)
        if ok:
            used = -(-old // page)
            for k in range(need):
                table[r, used + k] = free_pages[head + off + k]
            total[r] = old + new
            if need:
                taken = max(taken, off + need)
            for i in range(new):
                pg = int(table[r, (old + i) // page])
                positions[start + i] = old + i
                if 0 <= pg < num_pages:
                    slots[start + i] = pg * page + (old + i) % page
                else:
                    refused = True
        refused |= not ok
        off += need
    cu = np.minimum(cu, 2 ** 31 - 1)
    return table, cu, total, positions, slots, head + taken, refused

"""Cases of the serving operators: page tables and slot maps built on the GPU,
the 4-bit K/V cache's write and read-back, and attention over that cache.

Each case runs in a plain form (elementary torch operations in fp32) or, with
``own`` true, through the library's entry points.

The cache: uint8 [num_pages, h_kv, page_size / 16, chunk_bytes].  A chunk holds
16 tokens of one kv head: K codes (1024 bytes), V codes (1024 bytes), then the
f16 arrays K step, K minimum, V step, V minimum (32 bytes for each of the
128 / group groups, each).  An element stands for step * code + minimum.
"""
import math

import torch

own = False

D = 128                      # head dimension
CHUNK = 16                   # tokens of a chunk


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _attn(name, batch, max_len, max_q, h_q, h_kv, page, group, dtype, ragged, lens):
    c = {"op": "attn", "batch": batch, "max_len": max_len, "max_q": max_q, "h_q": h_q, "h_kv": h_kv, "page": page,
         "group": group, "dtype": dtype, "ragged_q": ragged, "lens": lens}
    return dict(c, name=name) if name else c


def _tables(name, batch, page, old_max, new_max, lens):
    c = {"op": "tables", "batch": batch, "page": page, "old_max": old_max, "new_max": new_max, "lens": lens}
    return dict(c, name=name) if name else c


def _write(name, tokens, h_kv, page, group, dtype, start, fused, pad):
    c = {"op": "write", "tokens": tokens, "h_kv": h_kv, "page": page, "group": group, "dtype": dtype, "start": start,
         "fused": fused, "pad": pad}
    return dict(c, name=name) if name else c


def _read(name, tokens, h_kv, page, group, dtype, start, out_page, pad):
    c = {"op": "read", "tokens": tokens, "h_kv": h_kv, "page": page, "group": group, "dtype": dtype, "start": start,
         "out_page": out_page, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's chat turn, one token at a time: nothing to hide latency behind
        _attn("decode one request", 1, 700, 1, 32, 8, 16, 64, "bf16", False, 1),
        # a full decode batch of requests of all ages
        _attn("decode batch of 64", 64, 16384, 1, 32, 4, 64, 32, "bf16", False, 2),
        # one request over a whole book: few rows, a very long axis
        _attn("decode at 256K", 1, 262144, 1, 32, 8, 64, 32, "bf16", False, 3),
        # a step that checks up to 8 drafted tokens of each request, e4m3 queries
        _attn("verify drafts, e4m3", 32, 8192, 8, 32, 8, 128, 64, "e4m3", True, 4),
        # an odd head layout, large pages, a batch padded with empty requests
        _attn("decode odd heads", 7, 5001, 1, 15, 5, 256, 128, "bf16", False, 5),
        # the tables of a decode step: one new token for each request
        _tables("tables of a decode step", 64, 64, 16384, 1, 6),
        # the tables when a batch of prompts is admitted
        _tables("tables of admitted prompts", 128, 16, 4097, 8192, 7),
        # a decode step's new keys and values
        _write("append 64 tokens", 64, 8, 64, 32, "bf16", 77, True, 0),
        # a long prompt's keys and values, straight from the fused projection
        _write("write a 64K prompt", 65536, 8, 64, 32, "bf16", 0, True, 0),
        # a prompt chunk held in e4m3, starting inside a page, in a padded buffer
        _write("write e4m3, odd", 5003, 5, 32, 128, "e4m3", 1001, False, 93),
        # a 128K prefix brought back into the bf16 pages of the prefill kernels
        _read("read a 128K prefix", 131072, 4, 64, 32, "bf16", 0, 64, 0),
        # a short prefix to contiguous e4m3
        _read("read e4m3, odd", 1501, 8, 16, 64, "e4m3", 333, 0, 35),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "tables", "write", "read"])
    page = rng.choice([16, 32, 64, 128, 256])
    group = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "e4m3"])
    seed = rng.randrange(1 << 20)
    if op == "tables":
        batch = _log(rng, 1, 1024)
        return _tables(None, batch, page, _log(rng, 1, 32768), _log(rng, 1, max(1, 1000000 // batch)), seed)
    h_kv = rng.randint(1, 8)
    if op == "attn":
        g = rng.randint(1, 16)
        batch = _log(rng, 1, 128)
        max_len = _log(rng, 16, min(262144, 2000000 // (batch * h_kv)))
        max_q = rng.choice([1, 1, 1, 2, 3, 4, 5, 6, 7, 8])
        max_q = max(1, min(max_q, 64000000 // (batch * h_kv * g * max_len)))
        return _attn(None, batch, max_len, max_q, g * h_kv, h_kv, page, group, dtype, max_q > 1 and rng.random() < 0.5,
                     seed)
    tokens = _log(rng, 1, 500000 // h_kv)
    start = rng.randint(0, 2000)
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    if op == "write":
        return _write(None, tokens, h_kv, page, group, dtype, start, rng.random() < 0.5, pad)
    return _read(None, tokens, h_kv, page, group, dtype, start, rng.choice([0, 16, 64, 128]), pad)


def _lengths(case):
    """Cached lengths and query counts of an attention case, or old and new
    lengths of a tables case: part of the case, not of its data."""
    g = torch.Generator().manual_seed(case["lens"])
    b = case["batch"]
    if case["op"] == "tables":
        old = torch.randint(0, case["old_max"] + 1, (b,), generator=g)
        new = torch.randint(1 if case["new_max"] == 1 else 0, case["new_max"] + 1, (b,), generator=g)
        return old, new
    lens = torch.randint(1, case["max_len"] + 1, (b,), generator=g)
    lens[0] = case["max_len"]
    lq = torch.full((b,), case["max_q"])
    if case["ragged_q"]:
        lq = torch.randint(1, case["max_q"] + 1, (b,), generator=g)
    lens = torch.maximum(lens, lq)
    if b > 4:
        lens[b // 2] = 0      # a request that has left the batch: its rows stay, its cache is empty
    return lens, lq


# ----------------------------------------------------------------------------
# the plain form of the 4-bit format
# ----------------------------------------------------------------------------

def _quantise(x, group):
    """fp32 [..., 128] -> codes uint8 [..., 128], step and minimum f16 [..., 128 / group]."""
    x = x.clamp(-65504.0, 65504.0).unflatten(-1, (D // group, group))
    lo = x.amin(-1).half()
    step = ((x.amax(-1) - lo.float()) / 15).clamp(0, 65504.0).half()
    s = step.float()
    inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    code = torch.round((x - lo.float().unsqueeze(-1)) * inv.unsqueeze(-1)).clamp(0, 15)
    return code.to(torch.uint8).flatten(-2), step, lo


def _values(code, step, lo, group):
    c = code.float().unflatten(-1, (D // group, group))
    return (c * step.float().unsqueeze(-1) + lo.float().unsqueeze(-1)).flatten(-2)


def _pair(c):
    """Nibbles [..., 2 n] -> bytes [..., n], the first in the low half."""
    c = c.unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4)


def _unpair(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _token_bytes(kc, ks, km, vc, vs, vm):
    """A token's bytes, [..., 128 + 1024 / group], in the order of _offsets."""
    k = _pair(kc.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3))          # [lane][quarter][8 dims]
    v = _pair(vc.unflatten(-1, (4, 8, 4)).transpose(-3, -2).flatten(-3))          # [row][quarter][4 dims]
    return torch.cat([k, v] + [x.contiguous().view(torch.uint8) for x in (ks, km, vs, vm)], -1)


def _offsets(group, device):
    """Byte offsets inside a chunk of each of its 16 tokens' bytes: int64 [16, 128 + 1024 / group]."""
    n = D // group
    t = torch.arange(CHUNK, device=device).view(CHUNK, 1)
    b = torch.arange(64, device=device).view(1, 64)
    k = t * 64 + b
    v = 1024 + (t // 8) * 512 + (b // 8) * 64 + (t % 8 // 2) * 16 + (t % 2) * 8 + b % 8
    g = torch.arange(2 * n, device=device).view(1, 2 * n)
    ks = 2048 + t * 2 * n + g
    vs = 2048 + 64 * n + (t % 8 // 2) * 8 * n + (g // 2) * 8 + (t // 8) * 4 + (t % 2) * 2 + g % 2
    return torch.cat([k, v, ks, ks + 32 * n, vs, vs + 32 * n], 1)


def _byte_index(slots, h_kv, page, group):
    """Where the bytes of the tokens at `slots` are in the cache: int64 [tokens, h_kv, bytes]."""
    off = _offsets(group, slots.device)
    slots = slots.long()
    size = 2048 + 128 * (D // group)
    head = torch.arange(h_kv, device=slots.device)
    chunk = ((slots // page).unsqueeze(1) * h_kv + head) * (page // CHUNK) + (slots % page // CHUNK).unsqueeze(1)
    return (chunk * size).unsqueeze(2) + off[slots % CHUNK].unsqueeze(1)


def _from_bytes(b, group):
    """Token bytes [..., 128 + 1024 / group] -> K and V values, fp32 [..., 128]."""
    n = D // group
    k = _unpair(b[..., :64]).unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3)
    v = _unpair(b[..., 64:128]).unflatten(-1, (8, 4, 4)).transpose(-3, -2).flatten(-3)
    m = b[..., 128:].contiguous().view(torch.float16)
    ks, km, vs, vm = m.split(n, -1)
    return _values(k, ks, km, group), _values(v, vs, vm, group)


def _pack_pages(k, v, group):
    """K and V values fp32 [pages, h_kv, page, 128] -> cache bytes."""
    kc, ks, km = _quantise(k, group)
    vc, vs, vm = _quantise(v, group)
    n = D // group
    p, h, ps = k.shape[:3]
    c = (p, h, ps // CHUNK)
    kb = _pair(kc.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3)).reshape(*c, 1024)
    vb = _pair(vc.unflatten(-1, (4, 8, 4)).transpose(-3, -2).flatten(-3)).reshape(*c, 2, 4, 2, 8, 8)
    vb = vb.permute(0, 1, 2, 3, 6, 4, 5, 7).reshape(*c, 1024)

    def rows(x):
        return x.reshape(*c, CHUNK * n).view(torch.uint8)

    def lanes(x):
        return x.reshape(*c, 2, 4, 2, n).permute(0, 1, 2, 4, 6, 3, 5).reshape(*c, CHUNK * n).view(torch.uint8)

    return torch.cat([kb, vb, rows(ks), rows(km), lanes(vs), lanes(vm)], -1)


def _unpack_pages(b, group):
    """Cache bytes [..., chunks, chunk_bytes] -> K and V values fp32 [..., chunks * 16, 128]."""
    n = D // group
    k = _unpair(b[..., :1024].unflatten(-1, (CHUNK, 64))).unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3)
    v = b[..., 1024:2048].unflatten(-1, (2, 8, 4, 2, 8)).movedim(-4, -2).flatten(-5, -3)   # [16 tokens, 8 rows, 8]
    v = _unpair(v).unflatten(-1, (4, 4)).transpose(-3, -2).flatten(-3)
    m = b[..., 2048:].contiguous().view(torch.float16).unflatten(-1, (4, CHUNK * n))
    ks, km = (m[..., i, :].unflatten(-1, (CHUNK, n)) for i in (0, 1))
    vs, vm = (m[..., i, :].unflatten(-1, (4, n, 2, 2)).movedim(-2, -4).movedim(-2, -1).flatten(-4, -2) for i in (2, 3))
    return _values(k, ks, km, group).flatten(-3, -2), _values(v, vs, vm, group).flatten(-3, -2)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _keys(shape, gen):
    """Keys as models have them: a few channels with large means, the rest near zero."""
    x = torch.randn(shape, generator=gen, device="cuda")
    bias = torch.randn((shape[1], 1, D) if len(shape) == 4 else (shape[1], D), generator=gen, device="cuda")
    return x + bias * bias.abs()


def _e4m3(x, dims):
    """fp32 -> e4m3 codes (uint8) and one scale for each head."""
    scale = x.abs().amax(dims) / 448
    shape = [1] * x.dim()
    shape[1] = -1
    return (x / scale.view(shape)).to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous()


def _pages_of(slots_needed, page, gen):
    """A shuffled page list that holds that many slots, and how many pages the pool has."""
    used = -(-slots_needed // page)
    pool = used + 3
    return torch.randperm(pool, generator=gen, device="cuda")[:used].to(torch.int32), pool


def _slot_map(case, gen):
    """Slots of `tokens` tokens that follow `start` earlier ones of their request, then the padding's -1."""
    pages, pool = _pages_of(case["start"] + case["tokens"], case["page"], gen)
    pos = torch.arange(case["start"], case["start"] + case["tokens"], device="cuda")
    slots = pages[pos // case["page"]].long() * case["page"] + pos % case["page"]
    pad = torch.full((case["pad"],), -1, device="cuda")
    return torch.cat([slots, pad]).to(torch.int32), pool


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "tables":
        old, new = _lengths(case)
        page = case["page"]
        used = -(-old // page)
        need = -(-(old + new) // page) - used
        pool = int((used + need).sum()) + 5
        width = int((used + need).max()) + 1
        order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((case["batch"], width), dtype=torch.int32, device="cuda")
        live = torch.arange(width).unsqueeze(0) < used.unsqueeze(1)
        table[live.cuda()] = order[:int(used.sum())]
        s.update(seqlens=old.to(torch.int32).cuda(), new_lens=new.to(torch.int32).cuda(), block_table=table, pool=pool,
                 free_pages=order, free_head=used.sum().view(1).to(torch.int32).cuda(),
                 capacity=max(1, int(new.sum()) + 7))
        return s
    h, group = case["h_kv"], case["group"]
    size = 2048 + 128 * (D // group)
    if op == "attn":
        lens, lq = _lengths(case)
        page = case["page"]
        count = -(-lens // page)
        pages, pool = _pages_of(max(1, int(count.sum())) * page, page, gen)
        width = max(1, int(count.max()))
        table = torch.zeros((case["batch"], width), dtype=torch.int32, device="cuda")
        live = torch.arange(width).unsqueeze(0) < count.unsqueeze(1)
        table[live.cuda()] = pages[:int(count.sum())]
        shape = (pool, h, page, D)
        s["cache"] = _pack_pages(_keys(shape, gen), torch.randn(shape, generator=gen, device="cuda"), group)
        cu = torch.cat([torch.zeros(1, dtype=torch.long), lq.cumsum(0)])
        q = torch.randn((int(cu[-1]), case["h_q"], D), generator=gen, device="cuda") * 1.5
        if case["dtype"] == "e4m3":
            s["q"], s["q_scale"] = _e4m3(q, (0, 2))
        else:
            s["q"], s["q_scale"] = q.to(torch.bfloat16), None
        s.update(block_table=table, seqlens_k=lens.to(torch.int32).cuda(),
                 cu=cu.to(torch.int32).cuda() if case["ragged_q"] else None)
        return s
    slots, pool = _slot_map(case, gen)
    s["slots"] = slots
    rows = slots.numel()
    if op == "write":
        if case["fused"]:      # keys and values inside the fused projection's rows
            qkv = torch.empty((rows, 4 * h, D), device="cuda")
            qkv.normal_(generator=gen)
            k, v = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
            k += torch.randn((h, D), generator=gen, device="cuda") * 2
        else:
            qkv, k, v = None, _keys((rows, h, D), gen), torch.randn((rows, h, D), generator=gen, device="cuda")
        if case["dtype"] == "e4m3":
            s["k"], s["k_scale"] = _e4m3(k, (0, 2))
            s["v"], s["v_scale"] = _e4m3(v, (0, 2))
        else:
            if case["fused"]:
                qkv = qkv.to(torch.bfloat16)
                k, v = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
            s.update(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16), k_scale=None, v_scale=None)
        s["cache"] = torch.zeros((pool, h, case["page"] // CHUNK, size), dtype=torch.uint8, device="cuda")
        s["k_out"] = torch.zeros((rows, h, D), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    shape = (pool, h, case["page"], D)
    s["cache"] = _pack_pages(_keys(shape, gen), torch.randn(shape, generator=gen, device="cuda"), group)
    out_rows, s["out_slots"] = rows, None
    if case["out_page"]:
        pages, out_pool = _pages_of(case["tokens"], case["out_page"], gen)
        pos = torch.arange(rows, device="cuda")
        pos = pos.clamp(max=case["tokens"] - 1)     # the padding rows read nothing, whatever their target
        s["out_slots"] = (pages[pos // case["out_page"]].long() * case["out_page"] + pos % case["out_page"]).to(torch.int32)
        out_rows = out_pool * case["out_page"]
    if case["dtype"] == "e4m3":
        s["k_scale"] = torch.rand(h, generator=gen, device="cuda") * 0.02 + 0.06
        s["v_scale"] = torch.rand(h, generator=gen, device="cuda") * 0.01 + 0.01
        s["k_out"] = torch.zeros((out_rows, h, D), dtype=torch.uint8, device="cuda")
    else:
        s["k_scale"] = s["v_scale"] = None
        s["k_out"] = torch.zeros((out_rows, h, D), dtype=torch.bfloat16, device="cuda")
    s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _as_values(x):
    """e4m3 codes as the values that they stand for (times their head's scale)."""
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def _run_own(s):
    from block_sparse_long_fp_gb300 import fprefill
    c, op = s["case"], s["case"]["op"]
    if op == "tables":
        if "plan" not in s:
            s["plan"] = fprefill.PageTables(s["block_table"], c["page"], s["pool"], s["capacity"])
        t = s["plan"].step(s["seqlens"], s["new_lens"], s["free_pages"], s["free_head"])
        return [s["block_table"], t.cu_seqlens_q, t.seqlens_k, t.positions, t.slots, t.free_head]
    if "plan" not in s:
        s["plan"] = fprefill.QCache(s["cache"], c["page"], c["group"])
    cache = s["plan"]
    if op == "attn":
        return list(cache.attn(s["q"], s["block_table"], s["seqlens_k"], cu_seqlens_q=s["cu"], max_q=c["max_q"],
                               q_scale=s["q_scale"]))
    if op == "write":
        cache.write(s["k"], s["v"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return list(cache.read(s["slots"], s["k_out"], s["v_out"]))
    cache.read(s["slots"], s["k_out"], s["v_out"], out_slots=s["out_slots"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return [_as_values(s["k_out"]), _as_values(s["v_out"])]


def _run_tables(s):
    page = s["case"]["page"]
    old, new = s["seqlens"].long(), s["new_lens"].long()
    table, free, head = s["block_table"], s["free_pages"], s["free_head"].long()
    total = old + new
    used = (old + page - 1) // page
    need = (total + page - 1) // page - used
    off = need.cumsum(0) - need
    p = torch.arange(table.shape[1], device=old.device).unsqueeze(0)
    k = p - used.unsqueeze(1)
    fresh = (k >= 0) & (k < need.unsqueeze(1))
    at = (head + off.unsqueeze(1) + k).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    ends = new.cumsum(0)
    i = torch.arange(s["capacity"], device=old.device)
    r = torch.searchsorted(ends, i, right=True).clamp(max=old.numel() - 1)
    pos = old[r] + i - (ends - new)[r]
    live = i < ends[-1]
    pos = torch.where(live, pos, torch.zeros_like(pos))
    slot = table[r, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    slot = torch.where(live, slot, torch.full_like(slot, -1))
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    return [table] + [x.to(torch.int32) for x in (cu, total, pos, slot, head + need.sum())]


def _decoded(x, scale):
    if scale is None:
        return x.float()
    return x.contiguous().view(torch.float8_e4m3fn).float() * scale.view(-1, 1)


def _run_attn(s):
    c = s["case"]
    b, h, g, lq, group = c["batch"], c["h_kv"], c["h_q"] // c["h_kv"], c["max_q"], c["group"]
    q = _decoded(s["q"], s["q_scale"])
    lens = s["seqlens_k"].long()
    if s["cu"] is None:
        first = torch.arange(b, device=lens.device) * lq
        count = torch.full_like(first, lq)
    else:
        first, count = s["cu"][:-1].long(), s["cu"][1:].long() - s["cu"][:-1].long()
    i = torch.arange(lq, device=lens.device)
    row = (first.unsqueeze(1) + i).clamp(max=q.shape[0] - 1)                      # [b, lq]
    here = i < count.unsqueeze(1)
    pos = lens.unsqueeze(1) - count.unsqueeze(1) + i                              # last key of each query
    pages = s["cache"][s["block_table"].long()]                                   # [b, pages, h, chunks, bytes]
    k, v = _unpack_pages(pages.transpose(1, 2).flatten(2, 3), group)              # [b, h, tokens, D]
    x = q[row].unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [b, h, lq * g, D]
    logit = torch.matmul(x, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    seen = torch.arange(k.shape[2], device=lens.device) <= pos.unsqueeze(2)       # [b, lq, tokens]
    seen = seen.repeat_interleave(g, 1).unsqueeze(1)
    logit = logit.masked_fill(~seen, -math.inf)
    top = logit.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    o = o.unflatten(2, (lq, g)).transpose(1, 2).flatten(2, 3)[here]               # [rows, h_q, D]
    lse = lse.unflatten(2, (lq, g)).transpose(1, 2).flatten(2, 3)[here]
    return [o.to(torch.bfloat16), lse.t().contiguous()]


def _run_write(s):
    c = s["case"]
    group, cache = c["group"], s["cache"].view(-1)
    kc, ks, km = _quantise(_decoded(s["k"], s["k_scale"]), group)
    vc, vs, vm = _quantise(_decoded(s["v"], s["v_scale"]), group)
    live = (s["slots"] >= 0).nonzero().squeeze(1)
    at = _byte_index(s["slots"][live], c["h_kv"], c["page"], group)
    cache[at] = _token_bytes(kc, ks, km, vc, vs, vm)[live]
    k, v = _from_bytes(cache[at], group)
    s["k_out"][live] = k.to(torch.bfloat16)
    s["v_out"][live] = v.to(torch.bfloat16)
    return [s["k_out"], s["v_out"]]


def _run_read(s):
    c = s["case"]
    live = (s["slots"] >= 0).nonzero().squeeze(1)
    at = _byte_index(s["slots"][live], c["h_kv"], c["page"], c["group"])
    k, v = _from_bytes(s["cache"].view(-1)[at], c["group"])
    to = live if s["out_slots"] is None else s["out_slots"][live].long()
    if s["k_scale"] is None:
        s["k_out"][to], s["v_out"][to] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        k = (k / s["k_scale"].view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v / s["v_scale"].view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["k_out"][to], s["v_out"][to] = k.view(torch.uint8), v.view(torch.uint8)
    return [_as_values(s["k_out"]), _as_values(s["v_out"])]


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _run_tables, "attn": _run_attn, "write": _run_write, "read": _run_read}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "tables":
        old, new = _lengths(case)
        need = int((-(-(old + new) // case["page"]) - -(-old // case["page"])).sum())
        partial = int(((old % case["page"] != 0) & (new > 0)).sum())
        t, b = int(new.sum()) + 7, case["batch"]
        return {"bytes": 8 * t + 16 * b + 8 * need + 4 * partial, "flops": 0}
    cached = 128 + 1024 // case["group"]
    if op == "attn":
        lens, lq = _lengths(case)
        e = 1 if case["dtype"] == "e4m3" else 2
        rows = int(lq.sum()) * case["h_q"]
        pairs = sum(max(0, n - k + i + 1) for n, k in zip(lens.tolist(), lq.tolist()) for i in range(k))
        return {"bytes": int(lens.sum()) * case["h_kv"] * cached + rows * (D * (e + 2) + 4) + 4 * case["batch"],
                "flops": 4 * D * case["h_q"] * pairs}
    e = 1 if case["dtype"] == "e4m3" else 2
    n = case["tokens"] * case["h_kv"]
    if op == "write":      # keys and values in, the cache out and in again, the values out
        return {"bytes": n * (2 * D * e + 2 * cached + 2 * D * 2) + 8 * case["tokens"], "flops": 0}
    return {"bytes": n * (cached + 2 * D * e) + 8 * case["tokens"], "flops": 0}


def _exact_rows(cache, page, group, slots, head):
    """K and V of one head at `slots`, in 64 bits, from the position of every nibble and f16 in a chunk."""
    n = D // group
    dim = torch.arange(D, device=slots.device)
    t = (slots % 16).unsqueeze(1)
    chunk = cache[slots // page, head, slots % page // 16]                        # [tokens, chunk_bytes]
    at_k = t * 64 + dim % 32 // 8 * 16 + dim // 32 * 4 + dim % 8 // 2
    at_v = 1024 + t // 8 * 512 + dim % 32 // 4 * 64 + t % 8 // 2 * 16 + t % 2 * 8 + dim // 32 * 2 + dim % 4 // 2
    ck, cv = (chunk.gather(1, at.expand(len(slots), D)).int() >> (dim % 2 * 4) & 15 for at in (at_k, at_v))
    f16 = chunk[:, 2048:].contiguous().view(torch.float16).double()               # [tokens, 4 * 16 * n]
    gk = t * n + dim // group
    gv = t % 8 // 2 * 4 * n + dim // group * 4 + t // 8 * 2 + t % 2
    k = ck.double() * f16.gather(1, gk) + f16.gather(1, gk + 16 * n)
    v = cv.double() * f16.gather(1, gv + 32 * n) + f16.gather(1, gv + 48 * n)
    return k, v


def _exact_attn(s):
    c = s["case"]
    h, g = c["h_kv"], c["h_q"] // c["h_kv"]
    lens, lq = _lengths(c)
    q = s["q"].double() if s["q_scale"] is None else s["q"].view(torch.float8_e4m3fn).double() * s["q_scale"].double().view(-1, 1)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["h_q"], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for r, (n, m) in enumerate(zip(lens.tolist(), lq.tolist())):
        t = torch.arange(n, device="cuda")
        slots = s["block_table"][r].long()[t // c["page"]] * c["page"] + t % c["page"] if n else t
        for head in range(h if n else 0):
            k, v = _exact_rows(s["cache"], c["page"], c["group"], slots, head)
            x = q[row:row + m, head * g:(head + 1) * g]
            z = (x.reshape(-1, D) @ k.t()).view(m, g, n) / math.sqrt(D)
            z = z.masked_fill((t > n - m + torch.arange(m, device="cuda").view(-1, 1)).unsqueeze(1), -math.inf)
            e = torch.logsumexp(z, -1, keepdim=True)
            out[row:row + m, head * g:(head + 1) * g] = (torch.exp(z - e).view(-1, n) @ v).view(m, g, D)
            lse[head * g:(head + 1) * g, row:row + m] = e.squeeze(-1).t()
        row += m
    return [out, lse]


def _exact_write(s):
    c = s["case"]

    def of(x, scale):
        x = x.double() if scale is None else x.contiguous().view(torch.float8_e4m3fn).double() * scale.double().view(-1, 1)
        x = x.view(*x.shape[:2], -1, c["group"])
        lo = x.min(-1, keepdim=True).values.half().double()
        step = ((x.max(-1, keepdim=True).values - lo).clamp(min=0) / 15).half().double()
        code = torch.where(step > 0, (x - lo) / step, 0.0).round().clamp(0, 15)
        y = (code * step + lo).flatten(2)
        return torch.where((s["slots"] >= 0).view(-1, 1, 1), y, 0.0)

    return [of(s["k"], s["k_scale"]), of(s["v"], s["v_scale"])]


def _exact_read(s):
    c = s["case"]
    outs = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    n = c["tokens"]
    to = torch.arange(n, device="cuda") if s["out_slots"] is None else s["out_slots"][:n].long()
    for head in range(c["h_kv"]):
        rows = _exact_rows(s["cache"], c["page"], c["group"], s["slots"][:n].long(), head)
        for x, y, scale in zip(outs, rows, (s["k_scale"], s["v_scale"])):
            x[to, head] = y if scale is None else y / scale[head].double()
    return outs


def exact(case, seed):
    if case["op"] == "tables":
        return None
    return {"attn": _exact_attn, "write": _exact_write, "read": _exact_read}[case["op"]](prepare(case, seed))

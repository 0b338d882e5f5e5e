"""Cases of the operators around the bf16 and e4m3 paged caches: rotary positions,
appending keys and values (rotated on the way) to the pages, and attention over
the pages from any position, one token to long chunks.

Each case runs in a plain form (elementary torch operations in fp32) or, with
``own`` true, through the library's entry points.

Rotary positions: with pairs (a, b) of dims -- (i, i + rot / 2), or (2 i, 2 i + 1)
where interleaved -- of the first `rot` dims of a head and the angle
t_i = position * inv_freq[i],
    a' = scale * (a cos t_i - b sin t_i),  b' = scale * (b cos t_i + a sin t_i)
(t_i negated for the inverse, which is the gradient too).  Dims from `rot` on stay.

The caches: [num_pages, page_size, h_kv, 128], bf16, or e4m3 codes that stand for
code * scale[head].
"""
import math

import torch

own = False

D = 128                      # head dimension


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _rope(name, tokens, heads, rot, layout, long, far, inverse, out, lens):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "rot": rot, "layout": layout, "long": long, "far": far,
         "inverse": inverse, "out": out, "lens": lens}
    return dict(c, name=name) if name else c


def _append(name, requests, new, start, h_q, h_kv, page, dtype, rot, layout, long, pad, lens):
    c = {"op": "append", "requests": requests, "new": new, "start": start, "h_q": h_q, "h_kv": h_kv, "page": page,
         "dtype": dtype, "rot": rot, "layout": layout, "long": long, "pad": pad, "lens": lens}
    return dict(c, name=name) if name else c


def _attn(name, batch, max_len, max_q, h_q, h_kv, page, dtype, q_dtype, ragged, lens):
    c = {"op": "attn", "batch": batch, "max_len": max_len, "max_q": max_q, "h_q": h_q, "h_kv": h_kv, "page": page,
         "dtype": dtype, "q_dtype": q_dtype, "ragged_q": ragged, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of one user, queries whose keys go to a cache of another form
        _rope("rotate one token", 1, 32, 128, "half", "smooth", 8191, False, "bf16", 1),
        # a long prompt's queries, frequencies scaled for contexts past the trained one
        _rope("rotate a 64K prompt", 65536, 32, 128, "half", "smooth", 0, False, "bf16", 2),
        # cached keys turned back (or the gradient of a rotation): part of the head, odd heads, far positions
        _rope("turn back, far and partial", 5003, 7, 64, "interleaved", "ramp", 1000000, True, "bf16", 3),
        # a decode step's new tokens: one for each of 64 requests
        _append("append 64 tokens", 64, 1, 16384, 32, 8, 64, "bf16", 128, "half", "smooth", 0, 4),
        # a long prompt's projections into the pages of the prefill kernels
        _append("append a 64K prompt", 1, 65536, 0, 32, 4, 64, "bf16", 128, "half", "none", 0, 5),
        # ragged prompts into e4m3 pages, an odd head layout, a padded batch
        _append("append to e4m3, odd", 9, 1001, 333, 15, 5, 256, "e4m3", 96, "interleaved", "linear", 93, 6),
        # one user's chat turn, one token at a time: nothing to hide latency behind
        _attn("decode one request", 1, 700, 1, 32, 8, 16, "bf16", "bf16", False, 7),
        # a full decode batch of requests of all ages
        _attn("decode batch of 64", 64, 16384, 1, 32, 4, 64, "bf16", "bf16", False, 8),
        # one request over a whole book, e4m3: few rows, a very long axis
        _attn("decode at 256K, e4m3", 1, 262144, 1, 32, 8, 64, "e4m3", "e4m3", False, 9),
        # a step that checks up to 8 drafted tokens of each request
        _attn("verify drafts", 32, 8192, 8, 32, 8, 128, "bf16", "bf16", True, 10),
        # a mixed step of a server: chunks of prompts beside decoding requests, e4m3 pages
        _attn("mixed step, e4m3", 12, 12000, 1024, 28, 4, 32, "e4m3", "bf16", True, 11),
        # a chunk of a prompt that starts at no block's border, behind 32K cached tokens
        _attn("chunk of 2048 behind 32K", 1, 34833, 2048, 32, 4, 64, "bf16", "bf16", False, 12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "e4m3"])
    layout = rng.choice(["half", "interleaved"])
    long = rng.choice(["none", "linear", "smooth", "ramp"])
    rot = rng.choice([128, 128, 128, 64, 32, 2 * rng.randint(1, 64)])
    seed = rng.randrange(1 << 20)
    h_kv = rng.randint(1, 8)
    g = rng.randint(1, 16)
    if op == "rope":
        heads = rng.randint(1, 64)
        return _rope(None, _log(rng, 1, 2000000 // heads), heads, rot, layout, long, rng.choice([0, _log(rng, 1, 4000000)]),
                     rng.random() < 0.3, dtype, seed)
    if op == "append":
        requests = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, 2000000 // (requests * (2 + g) * h_kv)))
        return _append(None, requests, new, _log(rng, 1, 131072), g * h_kv, h_kv, page, dtype, rot, layout, long,
                       rng.choice([0, 0, rng.randint(1, 40)]), seed)
    batch = _log(rng, 1, 128)
    max_len = _log(rng, 16, min(262144, 2000000 // (batch * h_kv)))
    max_q = rng.choice([1, 1, 1, rng.randint(2, 16), _log(rng, 17, 4096)])
    max_q = max(1, min(max_q, max_len, 1900000000 // (batch * h_kv * g * max_len)))
    return _attn(None, batch, max_len, max_q, g * h_kv, h_kv, page, dtype, rng.choice(["bf16", "e4m3"]),
                 max_q > 1 and rng.random() < 0.6, seed)


def _lengths(case):
    """Cached lengths (the new tokens included) and new tokens of each request: part of the case, not of its data."""
    g = torch.Generator().manual_seed(case["lens"])
    if case["op"] == "append":
        b = case["requests"]
        new = torch.full((b,), case["new"])
        if b > 1 and case["new"] > 1:
            new = torch.randint(1, case["new"] + 1, (b,), generator=g)
        return torch.randint(0, case["start"] + 1, (b,), generator=g) + new, new
    b = case["batch"]
    lens = torch.randint(1, case["max_len"] + 1, (b,), generator=g)
    lens[0] = case["max_len"]
    lq = torch.full((b,), case["max_q"])
    if case["ragged_q"]:
        lq = torch.randint(1, case["max_q"] + 1, (b,), generator=g)
        if case["max_q"] > 64:
            lq[b // 2 + 1:] = 1       # the decoding requests of a mixed step
    lens = torch.maximum(lens, lq)
    if b > 4:
        lens[b // 2] = 0              # a request that has left the batch: its rows stay, its cache is empty
    return lens, lq


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _frequencies(rot, long):
    """Radians a position for each pair, in 64 bits, and what cos and sin are multiplied by."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 500000.0 ** (-2 * i / rot)
    if long == "linear":
        return f / 8, 1.0
    if long == "smooth":       # long waves slowed 8 times, short ones kept, a blend between, by waves in 8192
        waves = 8192 * f / (2 * math.pi)
        keep = ((waves - 1) / 3).clamp(0, 1)
        return f * keep + f / 8 * (1 - keep), 1.0
    if long == "ramp":         # the same with a ramp over the pairs' indices, between 32 waves and 1 in 4096
        low, high = (rot * math.log(4096 / (w * 2 * math.pi)) / (2 * math.log(500000.0)) for w in (32, 1))
        low, high = max(0, math.floor(low)), min(rot - 1, math.ceil(high))
        slow = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / 16 * slow + f * (1 - slow), 0.1 * math.log(16) + 1
    return f, 1.0


def _keys(shape, gen):
    """Keys as models have them: a few channels with large means, the rest near zero."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    bias = torch.randn((shape[-2], D), generator=gen, device="cuda")
    return x.add_(bias * bias.abs())


def _e4m3(x, dims):
    """e4m3 codes (uint8) and one scale for each head."""
    scale = x.abs().amax(dims).float() / 448
    return (x.float() / scale.view(-1, 1)).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _table(lens, new, page, gen):
    """A shuffled block table int32 [batch, pages], the pool's pages; entries of no token's page are 0.  With `new`,
    only the pages of each request's last `new` tokens have a place in the pool."""
    count = -(-lens // page)
    first = torch.zeros_like(count) if new is None else (lens - new) // page
    used = int((count - first).sum())
    order = torch.randperm(used + 3, generator=gen, device="cuda").to(torch.int32)
    p = torch.arange(max(1, int(count.max()))).unsqueeze(0)
    live = (p >= first.unsqueeze(1)) & (p < count.unsqueeze(1))
    table = torch.zeros(live.shape, dtype=torch.int32, device="cuda")
    table[live.cuda()] = order[:used]
    return table, used + 3


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op != "attn":
        s["inv_freq"], s["factor"] = _frequencies(case["rot"], case["long"])
        s["freq"] = s["inv_freq"].cuda()
    if op == "rope":
        n, heads = case["tokens"], case["heads"]
        s["x"] = torch.empty((n, heads, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if case["far"]:
            s["positions"] = torch.randint(0, case["far"] + 1, (n,), generator=gen, device="cuda").to(torch.int32)
        else:
            s["positions"] = torch.arange(n, dtype=torch.int32, device="cuda")
        s["scale"] = None
        if case["out"] == "e4m3":
            s["scale"] = torch.rand(heads, generator=gen, device="cuda") * 0.005 + 0.012
        s["out"] = torch.empty((n, heads, D), dtype=torch.bfloat16 if s["scale"] is None else torch.uint8, device="cuda")
        return s
    h, h_q, page = case["h_kv"], case["h_q"], case["page"]
    lens, new = _lengths(case)
    if op == "append":
        table, pool = _table(lens, new, page, gen)
        n, pad = int(new.sum()), case["pad"]
        r = torch.repeat_interleave(torch.arange(len(new)), new)
        pos = torch.arange(n) - (new.cumsum(0) - new)[r] + (lens - new)[r]
        r, pos = r.cuda(), pos.cuda()
        slots = table[r, pos // page] * page + pos % page
        s["slots"] = torch.cat([slots, torch.full((pad,), -1, device="cuda")]).to(torch.int32)
        s["positions"] = torch.cat([pos, torch.zeros(pad, device="cuda")]).to(torch.int32)
        # queries, keys and values inside the fused projection's rows
        qkv = torch.empty((n + pad, h_q + 2 * h, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        qkv[:, h_q:h_q + h] += torch.randn((h, D), generator=gen, device="cuda") * 2
        s["q"], s["k"], s["v"] = qkv.split([h_q, h, h], 1)
        fp8 = case["dtype"] == "e4m3"
        kind = torch.uint8 if fp8 else torch.bfloat16
        s["k_cache"] = torch.zeros((pool, page, h, D), dtype=kind, device="cuda")
        s["v_cache"] = torch.zeros((pool, page, h, D), dtype=kind, device="cuda")
        s["q_out"] = torch.empty((n + pad, h_q, D), dtype=kind, device="cuda")
        for name, heads, low in (("q_scale", h_q, 0.012), ("k_scale", h, 0.03), ("v_scale", h, 0.012)):
            s[name] = torch.rand(heads, generator=gen, device="cuda") * 0.005 + low if fp8 else None
        return s
    s["block_table"], pool = _table(lens, None, page, gen)
    k = _keys((pool, page, h, D), gen)
    v = torch.empty((pool, page, h, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    s["k_scale"] = s["v_scale"] = s["q_scale"] = None
    if case["dtype"] == "e4m3":
        k, s["k_scale"] = _e4m3(k, (0, 1, 3))
        v, s["v_scale"] = _e4m3(v, (0, 1, 3))
    cu = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)])
    q = torch.empty((int(cu[-1]), h_q, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) * 1.5
    if case["q_dtype"] == "e4m3":
        q, s["q_scale"] = _e4m3(q, (0, 2))
    s.update(q=q, k_cache=k, v_cache=v, seqlens_k=lens.to(torch.int32).cuda(),
             cu=cu.to(torch.int32).cuda() if case["ragged_q"] else None)
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
    if op != "attn" and "rope" not in s:
        s["rope"] = fprefill.Rope(s["inv_freq"].tolist(), layout=c["layout"], scale=s["factor"])
    if op == "rope":
        return [_as_values(s["rope"].apply(s["x"], s["positions"], out=s["out"], out_scale=s["scale"],
                                           inverse=c["inverse"]))]
    if "cache" not in s:
        s["cache"] = fprefill.KVCache(s["k_cache"], s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    cache = s["cache"]
    if op == "append":
        q = cache.append(s["k"], s["v"], s["slots"], rope=s["rope"], positions=s["positions"], q=s["q"],
                         q_out=s["q_out"], q_scale=s["q_scale"])
        return [_as_values(x) for x in (q, s["k_cache"], s["v_cache"])]
    return list(cache.attn(s["q"], s["block_table"], s["seqlens_k"], cu_seqlens_q=s["cu"], max_q=c["max_q"],
                           q_scale=s["q_scale"]))


def _rotate(x, s, inverse=False):
    """x [tokens, heads, 128], rotated, in fp32 (angles in 64 bits)."""
    c = s["case"]
    rot = c["rot"]
    angle = (s["positions"].double().unsqueeze(1) * s["freq"]).unsqueeze(1)
    cos = (torch.cos(angle) * s["factor"]).float()
    sin = (torch.sin(angle) * (-s["factor"] if inverse else s["factor"])).float()
    x = x.float()
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _store(x, scale):
    """fp32 [.., heads, 128] as bf16, or as e4m3 codes."""
    if scale is None:
        return x.to(torch.bfloat16)
    return (x / scale.view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _run_rope(s):
    s["out"].copy_(_store(_rotate(s["x"], s, s["case"]["inverse"]), s["scale"]))
    return [_as_values(s["out"])]


def _run_append(s):
    n = s["slots"].numel() - s["case"]["pad"]
    at = s["slots"][:n].long()
    s["q_out"].copy_(_store(_rotate(s["q"], s), s["q_scale"]))
    s["k_cache"].view(-1, *s["k"].shape[1:])[at] = _store(_rotate(s["k"], s), s["k_scale"])[:n]
    s["v_cache"].view(-1, *s["v"].shape[1:])[at] = _store(s["v"].float(), s["v_scale"])[:n]
    return [_as_values(s[x]) for x in ("q_out", "k_cache", "v_cache")]


def _decoded(x, scale):
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * scale.view(-1, 1)


def _run_attn(s):
    c = s["case"]
    b, h, g, lq = c["batch"], c["h_kv"], c["h_q"] // c["h_kv"], c["max_q"]
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
    table = s["block_table"].long()
    k = _decoded(s["k_cache"][table].flatten(1, 2), s["k_scale"]).transpose(1, 2)           # [b, h, tokens, D]
    v = _decoded(s["v_cache"][table].flatten(1, 2), s["v_scale"]).transpose(1, 2)
    x = q[row].unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [b, h, lq * g, D]
    logit = torch.matmul(x, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    seen = torch.arange(k.shape[2], device=lens.device) <= pos.unsqueeze(2)       # [b, lq, tokens]
    logit = logit.masked_fill_(~seen.repeat_interleave(g, 1).unsqueeze(1), -math.inf)
    top = logit.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logit.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    o = o.unflatten(2, (lq, g)).transpose(1, 2).flatten(2, 3)[here]               # [rows, h_q, D]
    lse = lse.unflatten(2, (lq, g)).transpose(1, 2).flatten(2, 3)[here]
    return [o.to(torch.bfloat16), lse.t().contiguous()]


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _run_rope, "append": _run_append, "attn": _run_attn}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * D * (3 if case["out"] == "e4m3" else 4) + 4 * case["tokens"],
                "flops": 3 * case["rot"] * n}
    e = 1 if case["dtype"] == "e4m3" else 2
    lens, new = _lengths(case)
    h, h_q = case["h_kv"], case["h_q"]
    if op == "append":
        n, rows = int(new.sum()), int(new.sum()) + case["pad"]
        return {"bytes": (rows * h_q + n * 2 * h) * D * (2 + e) + 8 * rows,
                "flops": 3 * case["rot"] * (rows * h_q + n * h)}
    rows = int(new.sum()) * h_q
    eq = 1 if case["q_dtype"] == "e4m3" else 2
    pairs = 0
    for n, m in zip(lens.tolist(), new.tolist()):
        seen = min(m, max(0, n))                     # the rows that have a key: the last ones
        pairs += seen * (2 * n - seen + 1) // 2
    return {"bytes": int(lens.sum()) * h * 2 * D * e + rows * (D * (eq + 2) + 4) + 4 * case["batch"],
            "flops": 4 * D * h_q * pairs}


def _exact_rotation(s):
    """The rotation of a token as a 128 x 128 matrix for each token, in 64 bits, applied as one."""
    c = s["case"]
    rot = c["rot"]
    i = torch.arange(rot // 2, device="cuda")
    a, b = (i, i + rot // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    sign = -1.0 if c.get("inverse") else 1.0
    z = torch.polar(torch.full((len(s["positions"]), rot // 2), float(s["factor"]), dtype=torch.float64, device="cuda"),
                    sign * s["positions"].double().view(-1, 1) * s["freq"].view(1, -1))

    def of(x):
        y = x.double()
        w = torch.complex(y[:, :, a], y[:, :, b]) * z.unsqueeze(1)
        y[:, :, a], y[:, :, b] = w.real, w.imag
        return y
    return of


def _exact_rope(s):
    y = _exact_rotation(s)(s["x"])
    return [y if s["scale"] is None else y / s["scale"].double().view(-1, 1)]


def _exact_append(s):
    rotate = _exact_rotation(s)
    n = s["slots"].numel() - s["case"]["pad"]
    page = s["case"]["page"]
    at = s["slots"][:n].long()
    outs = [rotate(s["q"])]
    for x, cache in ((rotate(s["k"]), s["k_cache"]), (s["v"].double(), s["v_cache"])):
        y = torch.zeros(cache.shape, dtype=torch.float64, device="cuda")
        y[at // page, at % page] = x[:n]
        outs.append(y)
    scales = (s["q_scale"], s["k_scale"], s["v_scale"])
    return [y if f is None else y / f.double().view(-1, 1) for y, f in zip(outs, scales)]


def _exact_attn(s):
    c = s["case"]
    h, g, page = c["h_kv"], c["h_q"] // c["h_kv"], c["page"]
    lens, lq = _lengths(c)

    def head_of(x, scale, head):
        if scale is None:
            return x.double()
        return x.contiguous().view(torch.float8_e4m3fn).double() * scale[head].double()

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["h_q"], s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for r, (n, m) in enumerate(zip(lens.tolist(), lq.tolist())):
        t = torch.arange(n, device="cuda")
        pages = s["block_table"][r].long()[t // page] if n else t
        for head in range(h if n else 0):
            k = head_of(s["k_cache"][pages, t % page, head], s["k_scale"], head)
            v = head_of(s["v_cache"][pages, t % page, head], s["v_scale"], head)
            for j in range(head * g, (head + 1) * g):
                for i0 in range(0, m, 1024):                 # bounds the memory of a chunk's logits
                    i1 = min(m, i0 + 1024)
                    z = head_of(s["q"][row + i0:row + i1, j], s["q_scale"], j) @ k.t() / math.sqrt(D)
                    last = n - m + torch.arange(i0, i1, device="cuda").view(-1, 1)
                    z = z.masked_fill(t > last, -math.inf)
                    e = torch.logsumexp(z, -1, keepdim=True)
                    w = torch.where(e > -math.inf, torch.exp(z - e), 0.0)
                    out[row + i0:row + i1, j] = w @ v
                    lse[j, row + i0:row + i1] = e.squeeze(-1)
        row += m
    return [out, lse]


def exact(case, seed):
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](prepare(case, seed))

"""Rotary positions and the bf16 / e4m3 paged cache on the GPU against their
float64 oracle."""
import math

import numpy as np
import pytest

from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_long_fp_gb300 import build, fprefill
    build.build()
    return fprefill


def i32(x):
    import torch
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def f32(x):
    import torch
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).cuda()


def host(x):
    """A bf16 or fp32 tensor's values, or the values of e4m3 codes (without their scale)."""
    import torch
    if x.dtype in (torch.uint8, torch.float8_e4m3fn):
        return oc.e4m3_values(x.view(torch.uint8).cpu().numpy())
    return x.double().cpu().numpy()


def bf16(seed, *shape, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


# -- rotary positions -------------------------------------------------------------

FREQ = {"short": 10000.0 ** (-np.arange(64) / 64), "long": 500000.0 ** (-np.arange(64) / 64) / 7.3}


def close(got, want, reach, e4m3=False):
    """got, rounded once, against want computed from terms of size `reach` (|a| + |b| times the scale).

    cos and sin: the angle in half turns is an fp32 (2^-24 of a number up to 1, so pi 2^-24 radians), its
    64-bit fraction is cut at 2^-32 turns (2 pi 2^-32), sincospif is within 2 steps (2^-22) and the factor
    rounds once more (2^-24); a product and a sum of two terms round three times (3 2^-24).  Together below
    (3.2 + 0.1 + 4 + 1 + 3) 2^-24 < 2^-20 of the terms.  Then half a step of the output."""
    err = 2.0 ** -20 * reach
    if e4m3:
        want = np.clip(want, -448, 448)
        tol = err + np.maximum(2.0 ** -4 * (np.abs(want) + err), 2.0 ** -10)
    else:
        tol = err + 2.0 ** -8 * (np.abs(want) + err) + 2.0 ** -134
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


def reach_of(x, half, interleaved, scale):
    r = np.abs(np.array(x, np.float64))
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    r[:, :, a] = r[:, :, b] = abs(scale) * (r[:, :, a] + r[:, :, b])
    return r


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rows,heads,rot,far,inverse", [
    (1, 1, 128, 9, False), (1, 32, 128, 8191, False), (3, 7, 64, 100000, True), (257, 5, 96, 2 ** 31 - 1, False),
    (40, 13, 2, 1000, False), (33, 3, 74, 5000000, True), (64, 40, 126, 70000, False), (5, 64, 32, 300, True),
    (2500, 2, 128, 131072, False)])
def test_rope(fp, rows, heads, rot, far, inverse, layout, out):
    x = bf16(rows + rot, rows, heads, 128)
    rng = np.random.default_rng(rot)
    pos = rng.integers(0, far, rows, endpoint=True)
    pos[0] = far
    if rows > 2:
        pos[1], pos[2] = 0, -far                     # a negative position turns backwards
    f = FREQ["long"][:rot // 2]
    r = fp.Rope(f, layout, scale=1.25)
    scale = 0.004 + 0.01 * rng.random(heads) if out == "e4m3" else None
    y = r.apply(x, i32(pos), out_scale=None if scale is None else f32(scale), inverse=inverse)
    want = oc.rope(host(x), pos, f, layout == "interleaved", 1.25, inverse)
    reach = reach_of(host(x), rot // 2, layout == "interleaved", 1.25)
    if scale is not None:
        s = np.float32(scale).astype(np.float64)[:, None]
        want, reach = want / s, reach / s
    close(host(y), want, reach, scale is not None)
    if scale is None:                                # the dims behind the rotated ones are the very same
        assert np.array_equal(host(y)[..., rot:], host(x)[..., rot:])


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 44), ("half", 48), ("interleaved", 50)])
def test_rope_in_place_and_strided(fp, layout, rot):
    """Rows inside a wider buffer, rotated where they lie: the same bits, and nothing beside them moves."""
    import torch
    wide = bf16(3, 70, 11, 160)
    before = wide.clone()
    x = wide[:, 2:7, 16:144]
    pos = i32(np.arange(70) * 31)
    r = fp.Rope(FREQ["short"][:rot // 2], layout)
    want = r.apply(x.contiguous(), pos)
    out = bf16(4, 70, 9, 128)
    kept = out.clone()
    r.apply(x, pos, out=out[:, 1:6])
    assert torch.equal(out[:, 1:6], want) and torch.equal(out[:, 0], kept[:, 0]) and torch.equal(out[:, 6:], kept[:, 6:])
    assert r.apply(x, pos, out=x) is x
    assert torch.equal(x, want)
    before[:, 2:7, 16:144] = want
    assert torch.equal(wide, before)


def test_rope_inverse_is_the_gradient(fp):
    """<u, R x> = <R' u, x>, R' the inverse, and the difference quotient of the rotation along u is R u."""
    n, scale = 9, 1.5
    r = fp.Rope(FREQ["short"], scale=scale)
    pos = i32(np.arange(n) * 977)
    x, u = bf16(1, n, 3, 128), bf16(2, n, 3, 128)
    rx, ru = host(r.apply(x, pos)), host(r.apply(u, pos, inverse=True))
    # both sides carry one rounding of bf16 an element (2^-8 of values up to scale (|a| + |b|))
    tol = 2.0 ** -8 * (np.abs(host(u) * rx).sum() + np.abs(ru * host(x)).sum())
    assert abs((host(u) * rx).sum() - (ru * host(x)).sum()) <= tol
    h = 2.0 ** -3                                    # x + h u in bf16, the step taken from what it became
    moved = (x.float() + h * u.float()).to(x.dtype)
    step = host(moved) - host(x)
    quotient = host(r.apply(moved, pos)) - rx
    want = oc.rope(step, pos.cpu().numpy(), FREQ["short"], scale=scale)
    assert np.all(np.abs(quotient - want) <= 2.0 ** -8 * (np.abs(rx) + np.abs(host(r.apply(moved, pos)))) + 1e-5)


@pytest.mark.parametrize("layout,rot", [("half", 64), ("half", 20), ("interleaved", 20)])
def test_rope_keeps_what_is_not_finite_in_its_pair(fp, layout, rot):
    import torch
    x = bf16(5, 6, 2, 128)
    x[1, 0, 3], x[2, 1, rot - 1], x[3, 0, rot], x[4, 1, 127] = math.nan, math.inf, math.inf, math.nan
    f = FREQ["short"][:rot // 2]
    got = host(fp.Rope(f, layout).apply(x, i32([5, 6, 7, 8, 9, 10])))
    want = oc.rope(host(x), [5, 6, 7, 8, 9, 10], f, layout == "interleaved")
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    codes = fp.Rope(f, layout).apply(x, i32([5, 6, 7, 8, 9, 10]), out_scale=f32([0.01, 0.01]))
    assert np.array_equal(np.isnan(host(codes)), np.isnan(want))       # an infinity saturates
    torch.cuda.synchronize()


def test_rope_of_far_offsets(fp):
    """Rows past 2^31 elements."""
    import torch
    rows, heads = 70, 2
    wide = torch.zeros((rows, 40000000), dtype=torch.bfloat16, device="cuda")
    x = wide[:, :heads * 128].unflatten(1, (heads, 128))
    x.copy_(bf16(8, rows, heads, 128))
    pos = np.arange(rows) * 3
    r = fp.Rope(FREQ["short"])
    want = r.apply(x.contiguous(), i32(pos))
    r.apply(x, i32(pos), out=x)
    assert torch.equal(x, want)


def test_rope_refusals(fp):
    import torch
    r = fp.Rope(FREQ["short"])
    x, pos = bf16(1, 4, 2, 128), i32([0, 1, 2, 3])
    for bad in (dict(x=x.float()), dict(x=x[..., :64]), dict(x=x[0]), dict(x=x.cpu()), dict(positions=pos.long()),
                dict(positions=pos[:3]), dict(out=x[:3]), dict(out=torch.empty_like(x, dtype=torch.uint8)),
                dict(out_scale=f32([1.0])), dict(out_scale=f32([1.0, 1.0]), out=x), dict(x=x.transpose(0, 2)),
                dict(x=torch.empty((4, 2, 136), dtype=torch.bfloat16, device="cuda")[..., 4:132]),
                dict(x=x[:, :0])):
        with pytest.raises(fp.FprefillError):
            r.apply(**dict(dict(x=x, positions=pos), **bad))
    for bad in (dict(inv_freq=[]), dict(inv_freq=np.ones(65)), dict(inv_freq=[math.nan]), dict(inv_freq=[1.0], layout="x"),
                dict(inv_freq=[1.0], scale=math.inf), dict(inv_freq=np.ones((2, 2)))):
        with pytest.raises(fp.FprefillError):
            fp.Rope(**bad)
    assert r.apply(x[:0], pos[:0]).shape == (0, 2, 128)


# -- append ---------------------------------------------------------------------

def pages_of(fp, pages, page, h, dtype, seed=0, scales=None):
    """A cache of random codes, and copies of them on the host."""
    import torch
    g = torch.Generator().manual_seed(seed)
    shape = (pages, page, h, 128)
    if dtype == "bf16":
        k, v = (torch.randn(shape, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        return fp.KVCache(k, v), 1.0, 1.0
    k, v = ((torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            for _ in range(2))
    rng = np.random.default_rng(seed)
    ks, vs = (np.float32(0.01 + 0.02 * rng.random(h)) for _ in range(2))
    if scales:
        ks, vs = ks * np.float32(scales), vs * np.float32(scales)
    return fp.KVCache(k, v, f32(ks), f32(vs)), ks.astype(np.float64)[:, None], vs.astype(np.float64)[:, None]


@pytest.mark.parametrize("dtype,q_dtype", [("bf16", "bf16"), ("e4m3", "e4m3"), ("e4m3", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("rows,h_q,h,page,rot,layout", [
    (1, 1, 1, 16, 128, "half"), (1, 32, 8, 64, 128, "half"), (64, 32, 8, 64, 128, "interleaved"), (37, 15, 5, 256, 96, "half"),
    (300, 7, 1, 32, 20, "half"), (61, 0, 3, 16, 64, "interleaved"), (1200, 16, 2, 128, 0, "half"), (50, 28, 4, 384, 0, "half")])
def test_append(fp, rows, h_q, h, page, rot, layout, dtype, q_dtype):
    """Rows of a fused projection into shuffled slots, a quarter of them skipped; everything else stays as it was."""
    import torch
    pages = -(-(rows + 20) // page) + 1
    c, ks, vs = pages_of(fp, pages, page, h, dtype, 1)
    before = [x.clone() for x in (c.k_cache, c.v_cache)]
    qkv = bf16(2, rows, h_q + 2 * h, 128)
    q, k, v = qkv.split([h_q, h, h], 1)
    rng = np.random.default_rng(rows)
    slots = rng.permutation(pages * page)[:rows]
    slots[rng.permutation(rows)[:rows // 4]] = -1
    pos = rng.integers(0, 200000, rows)
    f = FREQ["long"][:rot // 2]
    rope = fp.Rope(f, layout, 1.1) if rot else None
    qs = np.float32(0.004 + 0.01 * rng.random(h_q)) if q_dtype == "e4m3" and h_q else None
    got = c.append(k, v, i32(slots), rope=rope, positions=i32(pos) if rot else None, q=q if h_q else None,
                   q_scale=None if qs is None else f32(qs))

    def turned(x):
        x = host(x)
        if not rot:
            return x, np.abs(x)
        return oc.rope(x, pos, f, layout == "interleaved", 1.1), reach_of(x, rot // 2, layout == "interleaved", 1.1)

    if h_q:
        s = 1.0 if qs is None else qs.astype(np.float64)[:, None]
        want, reach = turned(q)
        close(host(got), want / s, reach / s, qs is not None)
    else:
        assert got is None
    live = slots >= 0
    for cache, old, (want, reach), s in ((c.k_cache, before[0], turned(k), ks), (c.v_cache, before[1], (host(v), np.abs(host(v))), vs)):
        flat, was = cache.flatten(0, 1), old.flatten(0, 1)
        close(host(flat)[slots[live]], (want / s)[live], (reach / s)[live], dtype == "e4m3")
        other = np.setdiff1d(np.arange(pages * page), slots)
        assert torch.equal(flat[torch.as_tensor(other).cuda()], was[torch.as_tensor(other).cuda()])
    assert c.device_status() == 0


def test_append_equals_rope_then_copy(fp):
    """The fused rotation gives the bits of fp_rope; q in place."""
    import torch
    c, *_ = pages_of(fp, 9, 64, 4, "bf16")
    k, v, q = bf16(1, 200, 4, 128), bf16(2, 200, 4, 128), bf16(3, 200, 12, 128)
    r = fp.Rope(FREQ["long"])
    pos, slots = i32(np.arange(200) + 5000), i32(np.random.default_rng(1).permutation(576)[:200])
    want_q, want_k = r.apply(q, pos), r.apply(k, pos)
    assert c.append(k, v, slots, r, pos, q=q, q_out=q) is q
    assert torch.equal(q, want_q)
    assert torch.equal(c.k_cache.flatten(0, 1)[slots.long()], want_k)
    assert torch.equal(c.v_cache.flatten(0, 1)[slots.long()], v)


@pytest.mark.parametrize("slots,code", [([3, -1, 7], 0), ([3, -2, 7], 5), ([3, 128, 7], 5), ([3, 2 ** 31 - 1, -2 ** 31], 5)])
def test_append_leaves_out_slots_out_of_range(fp, slots, code):
    import torch
    c, *_ = pages_of(fp, 2, 64, 2, "bf16")
    before = c.k_cache.clone(), c.v_cache.clone()
    k, v, q = bf16(1, 3, 2, 128), bf16(2, 3, 2, 128), bf16(3, 3, 4, 128)
    r = fp.Rope(FREQ["short"])
    got = c.append(k, v, i32(slots), r, i32([7, 8, 9]), q=q)
    assert c.device_status() == code
    assert torch.equal(got, r.apply(q, i32([7, 8, 9])))
    rk = r.apply(k, i32([7, 8, 9]))
    for cache, x, old in ((c.k_cache, rk, before[0]), (c.v_cache, v, before[1])):
        want = old.flatten(0, 1).clone()
        for i, s in enumerate(slots):
            if 0 <= s < 128:
                want[s] = x[i]
        assert torch.equal(cache.flatten(0, 1), want)
    c.reset_status()
    assert c.device_status() == 0


def test_append_past_4_gb(fp):
    import torch
    page, h, pages = 128, 8, 20000                   # 5.2 GB each
    k = torch.zeros((pages, page, h, 128), dtype=torch.bfloat16, device="cuda")
    c = fp.KVCache(k, torch.zeros_like(k))
    x, y = bf16(1, 3, h, 128), bf16(2, 3, h, 128)
    last = pages * page - 1
    slots = [last, 2 ** 21 + 5, 7]
    c.append(x, y, i32(slots))
    at = torch.as_tensor(slots).cuda()
    assert torch.equal(c.k_cache.flatten(0, 1)[at], x) and torch.equal(c.v_cache.flatten(0, 1)[at], y)
    assert int((c.k_cache.flatten(0, 1).view(torch.int16) != 0).any(-1).any(-1).sum()) == 3


def test_append_refusals(fp):
    import torch
    c, *_ = pages_of(fp, 3, 16, 2, "bf16")
    k, q, slots, pos = bf16(1, 4, 2, 128), bf16(2, 4, 6, 128), i32([0, 1, 2, 3]), i32([0, 1, 2, 3])
    r = fp.Rope(FREQ["short"])
    good = dict(k=k, v=k, slots=slots)
    for bad in (dict(k=k[:3]), dict(v=k[:3]), dict(slots=slots[:3]), dict(slots=slots.long()), dict(rope=r), dict(positions=pos),
                dict(q_out=q), dict(q_scale=f32(np.ones(6))), dict(q=q[:3]), dict(q=q, q_out=q[:3]), dict(k=bf16(1, 4, 3, 128)),
                dict(q=q, q_scale=f32(np.ones(5))), dict(q=q, q_scale=f32(np.ones(6)), q_out=q), dict(rope=r, positions=pos[:2]),
                dict(k=k.float()), dict(q=q.cpu())):
        with pytest.raises(fp.FprefillError):
            c.append(**dict(good, **bad))
    x = torch.empty((3, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    for bad in ((x, x[:2]), (x.float(), x), (x, x, f32([1, 1])), (x.cpu(), x), (x[:, :8], x[:, :8]), (x.transpose(1, 2), x),
                (x.view(torch.uint8), x.view(torch.uint8), f32([1, 1]), f32([1, 1]))):
        with pytest.raises(fp.FprefillError):
            fp.KVCache(*bad)
    y = torch.empty((3, 48, 2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fp.FprefillError):
        fp.KVCache(y, y)
    assert c.append(k[:0], k[:0], slots[:0]) is None
    assert c.append(k[:0], k[:0], slots[:0], q=q[:0]).shape == (0, 6, 128)


def test_append_captured_and_replayed(fp):
    """A graph reads the slots and positions of the moment; a second stream and graph beside it."""
    import torch
    c, *_ = pages_of(fp, 4, 64, 2, "bf16")
    r = fp.Rope(FREQ["short"])
    k, v, q = bf16(1, 20, 2, 128), bf16(2, 20, 2, 128), bf16(3, 20, 8, 128)
    slots, pos, q_out = i32(np.arange(20)), i32(np.arange(20)), torch.empty_like(q)
    c.append(k, v, slots, r, pos, q=q, q_out=q_out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(k, v, slots, r, pos, q=q, q_out=q_out)
    slots.copy_(i32(np.arange(20) + 100))
    pos.copy_(i32(np.arange(20) + 3000))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.k_cache.flatten(0, 1)[100:120], r.apply(k, pos))
    assert torch.equal(q_out, r.apply(q, pos))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = r.apply(k, pos)
    s.synchronize()
    assert torch.equal(got, r.apply(k, pos))


# -- attention --------------------------------------------------------------------

def attn_case(fp, reqs, h_q, h, page, dtype, q_dtype, seed=0, spare=3, k_scale=1.0, q_scale=1.5, pad_rows=0):
    """Requests (length, queries) over a shuffled cache; what lies behind a request's last token is poison."""
    import torch
    rng = np.random.default_rng(seed)
    lens, lq = [n for n, _ in reqs], [m for _, m in reqs]
    count = [-(-n // page) for n in lens]
    pool = sum(count) + spare
    order = rng.permutation(pool)
    table = np.full((len(reqs), max(1, max(count)) + 1), -9, np.int64)
    at = 0
    for r, c in enumerate(count):
        table[r, :c] = order[at:at + c]
        at += c
    g = torch.Generator().manual_seed(seed)
    shape = (pool, page, h, 128)
    bias = torch.randn((h, 128), generator=g)
    k = torch.randn(shape, generator=g) * k_scale + bias * bias.abs() * k_scale
    v = torch.randn(shape, generator=g)
    used = torch.zeros((pool, page), dtype=torch.bool)
    for r, (n, c) in enumerate(zip(lens, count)):
        for j in range(c):
            used[table[r, j], :min(page, n - j * page)] = True
    total = sum(lq) + pad_rows
    q = torch.randn((total, h_q, 128), generator=g) * q_scale
    ks = vs = qs = None
    if dtype == "e4m3":
        ks, vs = (0.01 + 0.02 * torch.rand(h, generator=g) for _ in range(2))
        k, v = ((x / s.view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, s in ((k, ks), (v, vs)))
        k[~used], v[~used] = 0x7f, 0xff                                   # NaN
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        k[~used], v[~used] = math.nan, math.inf
    if q_dtype == "e4m3":
        qs = 0.01 + 0.02 * torch.rand(h_q, generator=g)
        q = (q / qs.view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        q = q.to(torch.bfloat16)
    up = [None if x is None else x.cuda() for x in (ks, vs, qs)]
    c = fp.KVCache(k.cuda(), v.cuda(), up[0], up[1])

    def values(x, s):
        return host(x) if s is None else host(x) * s.double().numpy()[:, None]
    cu = np.concatenate([[0], np.cumsum(lq)])
    return dict(c=c, q=q.cuda(), q_scale=up[2], table=table, lens=lens, lq=lq, cu=cu, qv=values(q, qs),
                kv=values(k, ks), vv=values(v, vs))


def reference(s, scale=None):
    """(out, lse, bound of out, bound of lse).

    A logit: 128 exact products summed in fp32, cut at 2^-23 of the partial sums a step: 2^-16 of the sum of
    their magnitudes at most; scaling and subtracting the maximum round at 2^-24 of the logit, the exponential
    is within 2^-22: d.  (bf16 queries of an e4m3 cache enter as two e4m3 terms, the largest in 2^7 .. 2^8: each
    element is exact, or off by half of e4m3's least step, 2^-10, so by 2^-17 of the row's largest.)  A weight is off by d, and by its rounding to bf16 (2^-8) or fp16 (2^-11): an output by
    that much of the weighted magnitudes of the values, then by fp32 sums of up to n terms cut at 2^-23 (a step
    sums 16, in 4 warps and several blocks), and by its own rounding (2^-8).  The LSE: d, a sum of n positive
    weights over 64 lanes and warps, and the rounding of itself."""
    out, lse = oc.attention(s["qv"], s["kv"], s["vv"], s["table"], s["lens"], s["lq"], scale)
    scale = 1 / math.sqrt(128) if scale is None else scale
    with np.errstate(invalid="ignore"):
        reach, _ = oc.attention(s["qv"], s["kv"], np.abs(s["vv"]), s["table"], s["lens"], s["lq"], scale)
    n = max(1, max(s["lens"]))
    kmax = np.abs(np.nan_to_num(s["kv"], nan=0.0, posinf=0.0)).max((0, 1))               # [h, 128]
    g = s["qv"].shape[1] // kmax.shape[0]
    size = scale * (np.abs(s["qv"]) * np.repeat(kmax, g, 0)).sum(-1)                      # [rows, h_q]
    d = 2.0 ** -16 * size + 2.0 ** -20
    if s["c"].k_scale is not None and s["q_scale"] is None:
        d = d + 2.0 ** -17 * scale * np.abs(s["qv"]).max(-1) * np.repeat(kmax.sum(-1), g)
    w = 2.0 ** -11 if s["c"].k_scale is not None else 2.0 ** -8
    tol = 2.0 ** -8 * np.abs(out) + reach * (w + 2 * d[..., None] + 2.0 ** -23 * (n / 16 + 64)) + 1e-30
    lse_tol = d.T + 2.0 ** -24 * (n / 64 + 64) + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
    return out, lse, tol, lse_tol


def check_attn(s, got, lse, scale=None, rows=None):
    want, want_lse, tol, lse_tol = reference(s, scale)
    n = sum(s["lq"]) if rows is None else rows
    got, lse = host(got)[:n], host(lse)[:, :n]
    bad = ~(np.abs(got - want[:n]) <= tol[:n])
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[:n][bad][:3], tol[:n][bad][:3])
    none = np.isneginf(want_lse[:, :n])
    assert np.array_equal(np.isneginf(lse), none)
    assert not got[none.T].any()
    assert np.all(np.abs(lse[~none] - want_lse[:, :n][~none]) <= lse_tol[:, :n][~none])


def run_attn(s, max_q=None, **kw):
    cu = i32(s["cu"])
    return s["c"].attn(s["q"], i32(s["table"]), i32(s["lens"]), cu_seqlens_q=cu, max_q=max_q or max(1, max(s["lq"])),
                       q_scale=s["q_scale"], **kw)


TYPES = [("bf16", "bf16"), ("e4m3", "e4m3"), ("e4m3", "bf16"), ("bf16", "e4m3")]


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("reqs,h_q,h,page", [
    ([(1, 1)], 1, 1, 16), ([(700, 1)], 32, 8, 16), ([(15, 1), (16, 1), (17, 1), (0, 1), (129, 1)], 8, 1, 128),
    ([(5001, 1), (64, 1), (0, 1), (1999, 1), (3, 1)], 15, 5, 256), ([(40000, 1)], 16, 2, 64),
    ([(300, 3), (2, 2), (1, 4), (0, 2), (90, 1)], 6, 2, 32), ([(1000, 8), (3000, 5), (8, 8)], 32, 8, 64),
    ([(2100, 4), (77, 1), (450, 2)], 48, 3, 16), ([(9000, 2), (33, 33), (500, 20)], 12, 3, 384),
    ([(130, 130), (1, 1)], 4, 4, 64), ([(100 + 37 * i, 1) for i in range(70)], 16, 4, 32)])
def test_attn(fp, reqs, h_q, h, page, dtype, q_dtype):
    s = attn_case(fp, reqs, h_q, h, page, dtype, q_dtype, seed=len(reqs) + h_q)
    out, lse = run_attn(s)
    check_attn(s, out, lse)
    assert s["c"].device_status() == 0
    again, lse2 = run_attn(s)                          # the same call gives the same bits
    assert bool((again == out).all()) and bool((lse2 == lse).all())


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("reqs,h_q,h,page", [
    ([(3000, 9), (1500, 1), (0, 1), (40, 2), (1100, 4), (1700, 1)], 32, 4, 64),       # drafts beside decodes
    ([(2000 + 300 * i, 5) for i in range(4)], 16, 2, 32),                             # as many each
    ([(2500, 300), (1200, 1), (1300, 1), (0, 1), (77, 2)], 16, 1, 16),                # a chunk, 16 heads share keys
    ([(4000, 200), (2600, 8), (1900, 9), (1, 1), (3100, 1)], 3, 3, 128),              # a chunk, none shared
    ([(1800 + i, 1 + i % 5) for i in range(40)], 9, 1, 64)])
def test_attn_rows_that_differ(fp, reqs, h_q, h, page, dtype, q_dtype):
    s = attn_case(fp, reqs, h_q, h, page, dtype, q_dtype, seed=len(reqs) + h_q)
    check_attn(s, *run_attn(s))
    check_attn(s, *run_attn(s, max_q=max(s["lq"]) + 7))
    assert s["c"].device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [1, 3, 7])
def test_attn_without_offsets_and_with_wider_bounds(fp, lq, dtype):
    """Equal rows need no offsets; a bound above the rows there are changes nothing beyond rounding."""
    import torch
    s = attn_case(fp, [(900, lq), (31, lq), (lq, lq)], 8, 2, 32, dtype, "bf16", seed=4)
    table, lens = i32(s["table"]), i32(s["lens"])
    out, lse = s["c"].attn(s["q"], table, lens)
    check_attn(s, out, lse)
    for bound in (lq, lq + 1, 20, 300):
        check_attn(s, *run_attn(s, max_q=bound))
    out, none = run_attn(s, want_lse=False)
    assert none is None
    given = torch.empty_like(out), torch.empty((8, 3 * lq), device="cuda")
    got = run_attn(s, out=given[0], lse=given[1])
    assert got[0] is given[0] and got[1] is given[1]
    check_attn(s, *got)
    scaled = run_attn(s, softmax_scale=0.2)
    check_attn(s, *scaled, scale=0.2)


def test_attn_strided_queries_and_rows_behind(fp):
    """Queries inside a fused projection; rows behind the last request's are left as they were."""
    import torch
    s = attn_case(fp, [(400, 2), (90, 1)], 8, 2, 64, "bf16", "bf16", seed=6, pad_rows=5)
    wide = torch.full((8, 14, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = s["q"]
    s["q"] = wide[:, 3:11]
    out = torch.full((8, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 8), 5.0, device="cuda")
    run_attn(s, out=out, lse=lse)
    check_attn(s, out, lse, rows=3)
    assert bool((out[3:] == 3).all()) and bool((lse[:, 3:] == 5).all())


@pytest.mark.parametrize("dtype,bad", [("bf16", math.nan), ("bf16", math.inf), ("e4m3", math.nan)])
@pytest.mark.parametrize("lq,h_q", [(2, 4), (9, 8), (40, 4)])
def test_attn_not_finite_reaches_only_rows_that_attend(fp, dtype, bad, lq, h_q):
    """A value that is not finite: its dim of the rows that attend it, no other.  In a key: the whole rows."""
    n, page, h = 230, 32, 2
    for at in (n - 1, n - lq + 1, n - lq, 17):         # the last token's, the second row's own, the first row's, a common one
        for side in ("v", "k"):
            s = attn_case(fp, [(n, lq), (50, 1)], h_q, h, page, dtype, "bf16", seed=at)
            c, name = s["c"], {"v": "vv", "k": "kv"}[side]
            cache = c.v_cache if side == "v" else c.k_cache
            pg = int(s["table"][0, at // page])
            cache[pg, at % page, 1, 77] = (0x7f if dtype == "e4m3" else bad)
            s[name][pg, at % page, 1, 77] = math.nan
            out, lse = run_attn(s)
            got = host(out)
            want, _ = oc.attention(s["qv"], s["kv"], s["vv"], s["table"], s["lens"], s["lq"])
            rows = np.arange(lq) + n - lq >= at                                  # that attend it
            hit = np.zeros(got.shape, bool)
            heads = slice(h_q // 2, h_q)
            if side == "v":
                hit[:lq, heads, 77] = rows[:, None]
            else:
                hit[:lq, heads] = rows[:, None, None]
            if side == "k" and math.isinf(bad):        # an infinite logit: the row is NaN, or the key counts for nothing
                assert np.isfinite(got[~hit]).all()
                continue
            assert np.array_equal(~np.isfinite(got), hit), (at, side)
            s2 = dict(s, vv=np.nan_to_num(s["vv"]), kv=np.nan_to_num(s["kv"]))
            ref, _, tol, _ = reference(s2)
            ok = ~hit
            assert np.all(np.abs(got - ref)[ok] <= tol[ok])


def test_attn_sharp_and_flat_rows(fp):
    """Logits of a thousand and of nothing, a maximum that rises token by token, values of large mean."""
    import torch
    for dtype in ("bf16", "e4m3"):
        s = attn_case(fp, [(3000, 1), (600, 4)], 8, 2, 64, dtype, "bf16", seed=9, k_scale=1.0, q_scale=30.0)
        check_attn(s, *run_attn(s))
        s = attn_case(fp, [(3000, 1), (600, 4)], 8, 2, 64, dtype, "bf16", seed=9, q_scale=0.0)
        check_attn(s, *run_attn(s))
    s = attn_case(fp, [(2000, 1)], 4, 1, 64, "bf16", "bf16", seed=3)
    t = torch.arange(2000)
    pages = torch.as_tensor(s["table"][0])[t // 64]
    ramp = (t.float() / 8).to(torch.bfloat16)
    s["c"].k_cache[pages.cuda(), (t % 64).cuda(), 0] = ramp[:, None].cuda() / 8
    s["c"].v_cache += 5
    s["kv"], s["vv"] = host(s["c"].k_cache), host(s["c"].v_cache)
    s["q"].fill_(0.25)
    s["qv"] = host(s["q"])
    check_attn(s, *run_attn(s))


def test_attn_bad_device_data(fp):
    """Pages out of range read as zeros, lengths out of range as an empty cache, rows outside q are left out."""
    s = attn_case(fp, [(200, 2), (90, 1)], 4, 2, 32, "bf16", "bf16", seed=5)
    c = s["c"]
    for bad in (-1, c.k_cache.shape[0], 2 ** 31 - 1):
        t = dict(s, table=s["table"].copy())
        t["table"][0, 2] = bad
        check_attn(t, *run_attn(t))
        assert c.device_status() == 5
        c.reset_status()
    for bad in (-1, s["table"].shape[1] * 32 + 1, 2 ** 31 - 1):
        t = dict(s, lens=[bad, 90])
        out, lse = run_attn(t)
        t["lens"] = [0, 90]
        check_attn(t, out, lse)
        assert c.device_status() == 5
        c.reset_status()
    for cu in ([0, 2, 9], [-3, 2, 3], [0, 2, 1], [5, 7, 9], [0, 2 ** 31 - 1, 3]):
        c.attn(s["q"], i32(s["table"]), i32(s["lens"]), cu_seqlens_q=i32(cu), max_q=2)
        c.device_status()
        c.reset_status()
    check_attn(s, *run_attn(s))
    assert c.device_status() == 0


def test_attn_refusals(fp):
    import torch
    s = attn_case(fp, [(200, 1), (90, 1)], 4, 2, 32, "bf16", "bf16", seed=5)
    c, table, lens = s["c"], i32(s["table"]), i32(s["lens"])
    good = dict(q=s["q"], block_table=table, seqlens_k=lens)
    q8 = s["q"].to(torch.float8_e4m3fn)
    for bad in (dict(q=s["q"][:, :3]), dict(q=s["q"].float()), dict(q=q8), dict(q_scale=f32([1] * 4)), dict(q=s["q"].cpu()),
                dict(block_table=table[:1]), dict(block_table=table.long()), dict(seqlens_k=lens[:1]),
                dict(cu_seqlens_q=i32([0, 1])), dict(max_q=0), dict(out=s["q"][:1]), dict(lse=f32(np.zeros((2, 4)))),
                dict(q=s["q"][:1]), dict(max_q=2), dict(q=q8, q_scale=f32([1] * 3))):
        with pytest.raises(fp.FprefillError):
            c.attn(**dict(good, **bad))
    out, lse = c.attn(s["q"][:0], table, lens, cu_seqlens_q=i32([0, 0, 0]))
    assert out.shape == (0, 4, 128) and lse.shape == (4, 0)


@pytest.mark.parametrize("lq", [2, 200])
def test_attn_past_4_gb(fp, lq):
    """A request whose last pages lie past 2^32 bytes of the cache."""
    import torch
    page, h, pages = 128, 8, 20000
    k = torch.zeros((pages, page, h, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = fp.KVCache(k, v)
    ids = [pages - 1, 3, pages - 2]
    for j, p in enumerate(ids):
        k[p], v[p] = bf16(j, page, h, 128), bf16(10 + j, page, h, 128)
    s = dict(c=c, q=bf16(30, lq, 16, 128), q_scale=None, table=np.array([ids]), lens=[300], lq=[lq], cu=np.array([0, lq]))
    small = np.array([[0, 1, 2]])
    s["qv"] = host(s["q"])
    out, lse = run_attn(s)
    at = torch.as_tensor(ids).cuda()
    check_attn(dict(s, table=small, kv=host(k[at]), vv=host(v[at])), out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_captured_two_graphs_and_streams(fp, dtype):
    """Graphs read the lengths and tables of the moment; two graphs, two streams and threads share nothing."""
    import threading
    import torch
    a = attn_case(fp, [(6000, 1), (90, 1), (0, 1)], 32, 8, 64, dtype, "bf16", seed=1)
    b = attn_case(fp, [(50, 1), (3000, 1), (777, 1)], 32, 8, 64, dtype, "bf16", seed=2)
    width = max(a["table"].shape[1], b["table"].shape[1])
    for s in (a, b):
        s["table"] = np.pad(s["table"], ((0, 0), (0, width - s["table"].shape[1])), constant_values=-1)
        run_attn(s)
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        table, lens, cu = i32(s["table"]), i32(s["lens"]), i32(s["cu"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s["c"].attn(s["q"], table, lens, cu_seqlens_q=cu, max_q=1)
        graphs.append((g, out, lens, table, cu))       # the graph reads them: they stay
    for _ in range(3):
        streams = [torch.cuda.Stream() for _ in graphs]
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, (_, out, *_) in zip((a, b), graphs):
            check_attn(s, *out)
    graphs[0][2].copy_(i32([5000, 64, 0]))
    graphs[0][0].replay()
    check_attn(dict(a, lens=[5000, 64, 0]), *graphs[0][1])
    results = [[], []]

    def work(s, got):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got.append(run_attn(s))
            torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=x) for x in zip((a, a), results)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for got in results:
        for out in got:
            check_attn(a, *out)


# -- requests of many rows --------------------------------------------------------

@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("reqs,h_q,h,page", [
    ([(128, 128)], 1, 1, 128), ([(65, 65)], 1, 1, 16), ([(700, 300)], 8, 1, 64), ([(129, 129), (1, 1), (0, 70), (40, 90)], 4, 2, 32),
    ([(5000, 17)], 16, 2, 256), ([(1000, 1000)], 6, 3, 16), ([(2111, 129), (64, 64), (3000, 1), (333, 100)], 14, 2, 384),
    ([(1500, 33), (900, 700)], 64, 2, 64), ([(20000, 130)], 4, 1, 32), ([(150 + 11 * i, 90 + i) for i in range(40)], 8, 4, 64)])
def test_attn_of_many_rows(fp, reqs, h_q, h, page, dtype, q_dtype):
    s = attn_case(fp, reqs, h_q, h, page, dtype, q_dtype, seed=len(reqs) + h_q)
    out, lse = run_attn(s)
    assert s["c"].device_status() == 0
    check_attn(s, out, lse)
    again, lse2 = run_attn(s)
    assert bool((again == out).all()) and bool((lse2 == lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_of_many_rows_without_keys(fp, dtype):
    """Requests that left the batch (all rows), and rows before the first key, of one half of a tile and of more."""
    for reqs in ([(0, 40)], [(0, 500), (700, 90), (0, 33)], [(30, 400), (1, 300), (0, 129)], [(0, 70)] * 5):
        s = attn_case(fp, reqs, 10, 2, 32, dtype, "bf16", seed=len(reqs))
        out, lse = run_attn(s)
        check_attn(s, out, lse)
        if len({m for _, m in reqs}) == 1:
            check_attn(s, *s["c"].attn(s["q"], i32(s["table"]), i32(s["lens"])))
        assert s["c"].device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_of_equal_rows_without_offsets(fp, dtype):
    s = attn_case(fp, [(900, 40), (331, 40), (40, 40)], 8, 2, 32, dtype, "bf16", seed=4)
    out, lse = s["c"].attn(s["q"], i32(s["table"]), i32(s["lens"]))
    check_attn(s, out, lse)
    for bound in (8, 16, 17, 400):                     # a bound that is too low changes nothing either
        check_attn(s, *run_attn(s, max_q=bound))
    assert s["c"].device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_of_many_rows_strided_and_rows_behind(fp, dtype):
    import torch
    s = attn_case(fp, [(400, 100), (90, 1)], 8, 2, 64, dtype, "bf16", seed=6, pad_rows=5)
    wide = torch.full((106, 14, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = s["q"]
    s["q"] = wide[:, 3:11]
    out = torch.full((106, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 106), 5.0, device="cuda")
    run_attn(s, out=out, lse=lse)
    check_attn(s, out, lse, rows=101)
    assert bool((out[101:] == 3).all()) and bool((lse[:, 101:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq,h_q", [(300, 2), (200, 16)])
def test_attn_of_many_rows_not_finite(fp, dtype, lq, h_q):
    """Values that are not finite at the diagonal, before it, and in several dims and blocks at once."""
    n, page, h = 1500, 64, 2
    s = attn_case(fp, [(n, lq)], h_q, h, page, dtype, "bf16", seed=3)
    hit = np.zeros((lq, h_q, 128), bool)
    for at, d in ((n - 1, 5), (n - lq, 6), (n - lq + 1, 7), (n - 150, 8), (n - 150, 127), (n - 100, 8), (100, 0), (n - lq - 1, 64)):
        pg = int(s["table"][0, at // page])
        s["c"].v_cache[pg, at % page, 1, d] = 0xff if dtype == "e4m3" else math.nan
        s["vv"][pg, at % page, 1, d] = math.nan
        hit[np.arange(lq) + n - lq >= at, h_q // 2:, d] = True
    out, _ = run_attn(s)
    got = host(out)
    assert np.array_equal(np.isnan(got), hit)
    ref, _, tol, _ = reference(dict(s, vv=np.nan_to_num(s["vv"])))
    assert np.all(np.abs(got - ref)[~hit] <= tol[~hit])


def test_attn_of_many_rows_sharp_and_flat(fp):
    for dtype in ("bf16", "e4m3"):
        for scale in (30.0, 0.0):
            s = attn_case(fp, [(700, 90), (600, 4)], 8, 2, 64, dtype, "bf16", seed=9, q_scale=scale)
            check_attn(s, *run_attn(s))


def test_attn_of_many_rows_bad_device_data(fp):
    s = attn_case(fp, [(300, 80), (90, 1)], 4, 2, 32, "bf16", "bf16", seed=5)
    c = s["c"]
    for bad in (-1, c.k_cache.shape[0], 2 ** 31 - 1):
        t = dict(s, table=s["table"].copy())
        t["table"][0, 2] = bad
        check_attn(t, *run_attn(t))
        assert c.device_status() == 5
        c.reset_status()
    for bad in (-1, s["table"].shape[1] * 32 + 1, 2 ** 31 - 1):
        t = dict(s, lens=[bad, 90])
        out, lse = run_attn(t)
        t["lens"] = [0, 90]
        check_attn(t, out, lse)
        assert c.device_status() == 5
        c.reset_status()
    for cu in ([0, 80, 90], [-3, 77, 81], [0, 81, 1], [5, 85, 81], [0, 2 ** 31 - 1, 3]):
        c.attn(s["q"], i32(s["table"]), i32(s["lens"]), cu_seqlens_q=i32(cu), max_q=80)
        assert c.device_status() in (0, 5)
        c.reset_status()
    check_attn(s, *run_attn(s))
    assert c.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_of_many_rows_captured(fp, dtype):
    import torch
    s = attn_case(fp, [(2000, 300), (90, 1), (500, 70)], 16, 4, 64, dtype, "bf16", seed=1)
    table, lens, cu = i32(s["table"]), i32(s["lens"]), i32(s["cu"])
    run_attn(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s["c"].attn(s["q"], table, lens, cu_seqlens_q=cu, max_q=300)
    for new in ([2000, 90, 500], [301, 64, 70], [1999, 0, 420]):
        lens.copy_(i32(new))
        g.replay()
        check_attn(dict(s, lens=new), *out)
    assert s["c"].device_status() == 0


def test_attn_of_both_query_types_on_one_cache(fp):
    """The scratch of a call depends on the queries' type too."""
    a = attn_case(fp, [(700, 200)], 8, 2, 64, "bf16", "bf16", seed=1)
    b = attn_case(fp, [(700, 200)], 8, 2, 64, "bf16", "e4m3", seed=1)
    for s in (a, b, a):
        check_attn(dict(s, c=a["c"]), *a["c"].attn(s["q"], i32(s["table"]), i32(s["lens"]), q_scale=s["q_scale"]))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq,h_q", [(2, 320), (40, 256), (70, 22)])
def test_attn_of_wide_groups(fp, dtype, lq, h_q):
    """More query heads a kv head than a tile's half has rows, as many, and a count that leaves rows over."""
    s = attn_case(fp, [(300, lq), (90, 1)], h_q, 2, 32, dtype, "bf16", seed=8)
    check_attn(s, *run_attn(s))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_of_many_requests(fp, dtype):
    """More requests than a block has threads, those of one row among those of many."""
    rng = np.random.default_rng(3)
    reqs = [(int(n), int(min(n, m))) for n, m in zip(rng.integers(0, 200, 900), rng.choice([1, 1, 1, 5, 40], 900))]
    s = attn_case(fp, reqs, 4, 2, 16, dtype, "bf16", seed=2)
    check_attn(s, *run_attn(s))
    s = attn_case(fp, [(int(n), 1) for n in rng.integers(0, 60, 4096)], 2, 1, 16, dtype, "e4m3", seed=2)
    check_attn(s, *run_attn(s))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [1, 60])
def test_attn_queries_that_are_not_finite(fp, dtype, lq):
    """Their rows, and no others."""
    s = attn_case(fp, [(400, lq), (90, 1)], 8, 2, 32, dtype, "bf16", seed=5)
    s["q"][0, 3, 17] = math.nan
    s["q"][lq, 1, 100] = math.inf
    s["q"][lq - 1, 6, 5] = -math.inf
    got, lse = run_attn(s)
    got, lse = host(got), host(lse)
    bad = np.zeros(got.shape[:2], bool)
    bad[0, 3] = True
    assert np.isnan(got[0, 3]).all() and np.isnan(lse[3, 0])
    bad[lq, 1] = bad[lq - 1, 6] = True                  # what an infinity makes of its row is not defined
    ref, ref_lse, tol, lse_tol = reference(dict(s, qv=np.nan_to_num(s["qv"])))
    assert np.all(np.abs(got - ref)[~bad] <= tol[~bad])
    assert np.all(np.abs(lse - ref_lse)[~bad.T] <= lse_tol[~bad.T])


def test_attn_after_a_wait_that_ran_out(fp):
    """A status of FP_ERR_TIMEOUT stays, and requests of many rows are left alone, until it is reset."""
    import torch
    s = attn_case(fp, [(500, 100), (90, 1)], 8, 2, 64, "bf16", "bf16", seed=5)
    out = torch.full((101, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    s["c"]._ws[0] = 6
    run_attn(s, out=out)
    assert s["c"].device_status() == 6
    assert bool((out[:100] == 3).all())
    s["c"].reset_status()
    check_attn(s, *run_attn(s, out=out))
    assert s["c"].device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [3, 40])
def test_attn_over_a_long_axis(fp, dtype, lq):
    """262144 tokens: few rows over all SMs, sums of many parts."""
    s = attn_case(fp, [(262144, lq)], 4, 1, 64, dtype, "bf16", seed=3, k_scale=0.3)
    check_attn(s, *run_attn(s))


@pytest.mark.parametrize("what", ["append", "columns", "tiles"])
def test_first_call_of_a_process_is_captured(what):
    """No call needs one before it outside the graph."""
    import os
    import subprocess
    import sys
    code = """
import torch
from block_sparse_long_fp_gb300 import fprefill as fp
k, v = (torch.randn(8, 64, 2, 128, device="cuda").bfloat16() for _ in range(2))
c, r, q = fp.KVCache(k, v), fp.Rope([1.0, 0.1]), torch.randn(300, 8, 128, device="cuda").bfloat16()
slots = torch.arange(300, dtype=torch.int32, device="cuda")
table, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8), torch.tensor([300], dtype=torch.int32, device="cuda")
cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
what = %r
def call():
    if what == "append":
        return c.append(q[:, :2], q[:, 2:4], slots, r, slots, q=q)
    return c.attn(q[:1] if what == "columns" else q, table, lens, max_q=1 if what == "columns" else 300)[0]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = call()
g.replay()
torch.cuda.synchronize()
assert torch.equal(a, call()) and c.device_status() == 0
""" % what
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_attn_two_streams_of_many_rows(fp):
    """Calls on two streams, and threads on one, have scratch of their own or one after the other."""
    import threading
    import torch
    a = attn_case(fp, [(3000, 100), (90, 1), (700, 300)], 16, 4, 64, "e4m3", "bf16", seed=1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], [], [], []]

    def work(i):
        with torch.cuda.stream(streams[i % 2]):
            for _ in range(4):
                got[i].append(run_attn(a))
            streams[i % 2].synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for outs in got:
        for o in outs:
            check_attn(a, *o)


# -- together ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompts_then_decode_steps(fp, dtype):
    """Tables, append with rotation, attention: two prompts, whose attention the prefill kernels compute too, a
    chunk that starts inside a block, then decode steps replayed from a graph."""
    import torch
    h_q, h, page, pool = 8, 2, 32, 64
    prompts, steps = [300, 77], 5
    f = FREQ["long"]
    rope = fp.Rope(f)
    fp8 = dtype == "e4m3"
    kind = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = (torch.zeros((pool, page, h, 128), dtype=kind, device="cuda") for _ in range(2))
    ks, vs, qs = (f32(np.full(n, 0.02)) if fp8 else None for n in (h, h, h_q))
    cache = fp.KVCache(kc, vc, ks, vs)
    table = i32(np.zeros((2, 20)))
    free = i32(np.random.default_rng(0).permutation(pool))
    lens, head = i32([0, 0]), i32([0])
    done = [0, 0]
    seed = [100]
    qs_all, keep = [], []

    def rows(n):
        seed[0] += 1
        return bf16(seed[0], n, h_q + 2 * h, 128).split([h_q, h, h], 1)

    def step(new, graph=None):
        nonlocal lens, head
        n = sum(new)
        t = fp.PageTables(table, page, pool, n)
        t.step(lens, i32(new), free, head)
        q, k, v = rows(n)
        q = cache.append(k, v, t.slots, rope, t.positions, q=q, q_scale=qs)
        out, lse = cache.attn(q, table, t.seqlens_k, cu_seqlens_q=t.cu_seqlens_q, max_q=max(new), q_scale=qs)
        lens, head = t.seqlens_k.clone(), t.free_head.clone()
        for r in range(2):
            done[r] += new[r]
        assert t.device_status() == 0 and cache.device_status() == 0
        return q, out, lse

    def check(new, q, out, lse):
        s = dict(c=cache, q=q, q_scale=qs, table=table.cpu().numpy(), lens=list(done), lq=new, cu=np.concatenate([[0], np.cumsum(new)]))
        scale = 0.02 if fp8 else 1.0
        s["qv"], s["kv"], s["vv"] = host(q) * scale, host(kc) * scale, host(vc) * scale
        check_attn(s, out, lse)

    q, out, lse = step(prompts)
    check(prompts, q, out, lse)
    layer = fp.Layer(q, kc, vc, table, [0, 300, 377], prompts, [0, 0], h_q, h, dtype=dtype, q_scale=qs, k_scale=ks, v_scale=vs)
    prefill, prefill_lse = layer.dense_attn()
    # both within a rounding of bf16 (2^-8) of outputs up to 4; the prefill's e4m3 weights add 2^-4 of theirs
    bound = 4 * 2.0 ** -7 + (2.0 ** -4 * 2 if fp8 else 0)
    assert float((prefill.float() - out.float()).abs().max()) <= bound
    assert float((prefill_lse - lse).abs().max()) <= 1e-2
    new = [100, 3]
    check(new, *step(new))                                 # from positions 300 and 77
    # decode: one graph, its inputs overwritten in place
    t = fp.PageTables(table, page, pool, 2)
    t.seqlens_k.copy_(lens)
    t.free_head.copy_(head)
    qkv, ones = bf16(7, 2, h_q + 2 * h, 128), i32([1, 1])
    qd, kd, vd = qkv.split([h_q, h, h], 1)

    def decode():
        t.step(t.seqlens_k, ones, free, t.free_head)
        q = cache.append(kd, vd, t.slots, rope, t.positions, q=qd, q_scale=qs)
        return (q, *cache.attn(q, table, t.seqlens_k, q_scale=qs))
    saved = t.seqlens_k.clone(), t.free_head.clone(), table.clone()
    decode()                                               # first calls are not captured
    t.seqlens_k.copy_(saved[0])
    t.free_head.copy_(saved[1])
    table.copy_(saved[2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, out, lse = decode()
    for i in range(steps):
        qkv.copy_(bf16(50 + i, 2, h_q + 2 * h, 128))
        g.replay()
        done[0], done[1] = done[0] + 1, done[1] + 1
        assert t.seqlens_k.tolist() == done
        check([1, 1], q, out, lse)
        if not fp8:
            close(host(q), oc.rope(host(qd), np.array(done) - 1, f), reach_of(host(qd), 64, False, 1.0))


def test_rotated_keys_into_the_4_bit_cache(fp):
    """A rope of its own beside a cache of another form, and keys turned back from it."""
    import torch
    c = fp.QCache.empty(8, 64, 2, 32)
    c.data.zero_()
    rope = fp.Rope(FREQ["short"])
    k, v, pos, slots = bf16(1, 90, 2, 128), bf16(2, 90, 2, 128), i32(np.arange(90) + 1000), i32(np.random.default_rng(0).permutation(512)[:90])
    c.write(rope.apply(k, pos), v, slots)
    back, _ = c.read(slots)
    again = rope.apply(back, pos, inverse=True)
    # a group of 32 rotated dims spans up to 2 * 1.5 * 4.5; a code is within 1 / 30 of that, two dims meet, bf16 rounds thrice
    span = 2 * 1.5 * 4.5
    assert float((again.float() - k.float()).abs().max()) <= 2 * span / 30 + 3 * 2.0 ** -8 * span

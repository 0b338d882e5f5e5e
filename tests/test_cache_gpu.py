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

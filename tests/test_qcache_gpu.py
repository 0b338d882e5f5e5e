"""The serving operators on the GPU against their float64 oracle: page tables,
the 4-bit cache's write and read, attention over it, and a run of them
together with the prefill kernels."""
import numpy as np
import pytest

from oracle import qcache as oq

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


# -- page tables ----------------------------------------------------------------

def tables_case(seed, batch, old_max, new_max, page, spare=3, pad=5, head=2):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, old_max + 1, batch)
    new = rng.integers(0, new_max + 1, batch)
    used, total = -(-old // page), -(-(old + new) // page)
    pool = int(total.sum()) + spare + head
    order = rng.permutation(pool)
    table = np.full((batch, max(1, int(total.max())) + 1), -7, np.int64)
    at = 0
    for r in range(batch):
        table[r, :used[r]] = order[at:at + used[r]]
        at += used[r]
    free = np.concatenate([order[:head], order[at:]])
    return table, old, new, free, pool, max(1, int(new.sum()) + pad)


def check_tables(fp, table, old, new, free, head, page, pool, capacity, in_place=False):
    import torch
    want = oq.page_tables(table, old, new, free, head, page, pool, capacity)
    bt = i32(table)
    p = fp.PageTables(bt, page, pool, capacity)
    lens, heads = i32(old), i32([head])
    if in_place:
        p.seqlens_k.copy_(lens)
        p.free_head.copy_(heads)
        lens, heads = p.seqlens_k, p.free_head
    p.step(lens, i32(new), i32(free), heads)
    for name, got, ref in zip(("table", "cu", "seqlens_k", "positions", "slots", "free_head"),
                              (bt, p.cu_seqlens_q, p.seqlens_k, p.positions, p.slots, p.free_head), want):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(ref)), ref), name
    assert (p.device_status() != 0) == bool(want[6])
    torch.cuda.synchronize()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,old_max,new_max,page", [
    (1, 0, 1, 16), (1, 0, 5000, 16), (5, 300, 0, 64), (64, 3000, 1, 64), (7, 100, 900, 256), (300, 50, 40, 32),
    (1500, 20, 9, 16), (4096, 6, 3, 128), (3, 70000, 40000, 128), (40, 2000, 3000, 384)])
def test_page_tables(fp, batch, old_max, new_max, page, in_place):
    table, old, new, free, pool, cap = tables_case(batch + page, batch, old_max, new_max, page)
    check_tables(fp, table, old, new, free, 2, page, pool, cap, in_place)


def test_page_tables_refuse_what_they_cannot_serve(fp):
    table, old, new, free, pool, cap = tables_case(11, 9, 200, 100, 16)
    check_tables(fp, table, old, new, free[:len(free) // 2], 2, 16, pool, cap)      # the free list runs out
    check_tables(fp, table, old, new, free[:0], 0, 16, pool, cap)
    check_tables(fp, table, old, new, free, len(free) + 4, 16, pool, cap)
    check_tables(fp, table, old, new, free, -1, 16, pool, cap)
    check_tables(fp, table, old, new, free, 2, 16, pool, max(1, cap // 2))          # the slot map runs out
    check_tables(fp, table[:, :8], old, new, free, 2, 16, pool, cap)                # the table is too narrow
    for at, value in ((0, -5), (4, -1)):
        bad = old.copy()
        bad[at] = value
        check_tables(fp, table, bad, new, free, 2, 16, pool, cap)
        bad = new.copy()
        bad[at] = value
        check_tables(fp, table, old, bad, free, 2, 16, pool, cap)
    bad = free.copy()
    bad[5] = pool
    check_tables(fp, table, old, new, bad, 2, 16, pool, cap)                        # page ids out of range
    big = new.copy()
    big[2] = 2 ** 31 - 1
    check_tables(fp, table, old, big, free, 2, 16, pool, cap)
    # lengths that an int cannot hold, though the table's pages could
    two = np.array([[0, 0, 0, 0]] * 2)
    check_tables(fp, two, np.array([2 ** 31 - 1, 2 ** 31 - 2]), np.array([1, 1]), np.array([0]), 0, 2 ** 30, 1, 4)


# -- write and read ---------------------------------------------------------------

def source(seed, rows, h, dtype, scale=1.0):
    """(tensor for the library, fp32 values it stands for, head scales or None)."""
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(rows, h, 128)).astype(np.float32) * scale + rng.normal(size=(h, 128)))
    if dtype == "bf16":
        x = x.to(torch.bfloat16)
        return x.cuda(), x.float().numpy(), None
    s = torch.from_numpy((0.01 + 0.01 * rng.random(h)).astype(np.float32))
    c = (x / s.view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).cuda(), (c.float() * s.view(-1, 1)).numpy(), s.cuda()


def some_slots(seed, rows, slots, skip=0):
    rng = np.random.default_rng(seed)
    s = rng.permutation(slots)[:rows]
    if skip:
        s[rng.permutation(rows)[:skip]] = -1
    return s


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,h,page", [(1, 1, 16), (3, 5, 32), (61, 2, 64), (40, 3, 256)])
def test_write_is_the_definition_bit_for_bit(fp, rows, h, page, group, dtype):
    import torch
    pages = -(-(rows + 20) // page) + 1
    data = np.random.default_rng(7).integers(0, 256, (pages, h, page // 16, oq.chunk_bytes(group)), dtype=np.uint8)
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    k, k32, ks = source(1, rows, h, dtype)
    v, v32, vs = source(2, rows, h, dtype, 0.3)
    slots = some_slots(3, rows, pages * page, skip=rows // 4)
    c.write(k, v, i32(slots), ks, vs)
    oq.write(data, page, group, slots, k32, v32)
    assert np.array_equal(c.data.cpu().numpy(), data)
    assert c.device_status() == 0


@pytest.mark.parametrize("group", [32, 128])
def test_write_of_whole_chunks_from_strided_rows(fp, group):
    """A prompt's consecutive slots (whole chunks, a ragged start and end), its
    keys and values inside wider rows."""
    import torch
    h, page, rows = 3, 64, 203
    data = np.zeros((6, h, 4, oq.chunk_bytes(group)), np.uint8)
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    x, x32, _ = source(5, rows, 5 * h, "bf16")
    pages = np.array([4, 0, 5, 2])
    pos = np.arange(13, 13 + rows)
    slots = pages[pos // page] * page + pos % page
    c.write(x[:, h:2 * h], x[:, 4 * h:], i32(slots))
    oq.write(data, page, group, slots, x32[:, h:2 * h], x32[:, 4 * h:])
    assert np.array_equal(c.data.cpu().numpy(), data)
    # the same rows one by one give the same cache
    d = fp.QCache(torch.zeros_like(c.data), page, group)
    for i in range(0, rows, 7):
        d.write(x[i:i + 7, h:2 * h], x[i:i + 7, 4 * h:], i32(slots[i:i + 7]))
    assert torch.equal(c.data, d.data)


def mixed_slots(seed, rows, pages, page):
    """Slots of many sequences laid end to end: prompts that start anywhere in a
    page, single tokens, padding, whole chunks that begin at any row."""
    rng = np.random.default_rng(seed)
    order = list(rng.permutation(pages))
    out = []
    while len(out) < rows:
        kind = rng.integers(0, 4)
        n = int(rng.integers(1, 4 if kind == 0 else 6 * page if kind == 1 else 40))
        if kind == 2:
            out += [-1] * n
            continue
        start = int(rng.integers(0, page)) if kind != 3 else 0
        need = -(-(start + n) // page)
        if need > len(order):
            out += [-1] * (rows - len(out))
            break
        mine = [order.pop() for _ in range(need)]
        out += [int(mine[p // page]) * page + p % page for p in range(start, start + n)]
    return np.array(out[:rows])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,h,page,seed", [(4103, 4, 16, 1), (2401, 7, 64, 2), (16400, 1, 128, 3), (2048, 8, 32, 4)])
def test_many_rows(fp, rows, h, page, seed, group, dtype):
    """Enough rows for the kernels that take 16 at a time, bit for bit: written,
    what no row names left alone, read back to mapped and to plain rows."""
    import torch
    pages = rows // page + 40
    slots = mixed_slots(seed, rows, pages, page) if seed != 4 else np.arange(rows) + 5 * page   # whole chunks in order
    data = np.random.default_rng(seed).integers(0, 256, (pages, h, page // 16, oq.chunk_bytes(group)), dtype=np.uint8)
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    x, x32, ks = source(seed, rows, 3 * h, dtype)
    k, v = x[:, :h], x[:, 2 * h:]
    scales = (None, None) if ks is None else (ks[:h].contiguous(), ks[2 * h:].contiguous())
    c.write(k, v, i32(slots), *scales)
    oq.write(data, page, group, slots, x32[:, :h], x32[:, 2 * h:])
    assert np.array_equal(c.data.cpu().numpy(), data)
    to = np.random.default_rng(seed + 1).permutation(rows + 7)[:rows]
    for target in (None, to):
        n = rows if target is None else rows + 7
        out = [torch.full((n, h, 128), 3, dtype=x.dtype, device="cuda") for _ in range(2)]
        want = [o.cpu().clone() for o in out]
        c.read(i32(slots), *out, out_slots=None if target is None else i32(target), k_scale=scales[0], v_scale=scales[1])
        live = slots >= 0
        at = torch.from_numpy((np.arange(rows) if target is None else target)[live])
        for w, val, s in zip(want, oq.read(data, page, group, slots), scales):
            y = torch.from_numpy(val).float()
            y = y.bfloat16() if s is None else (y / s.cpu().view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            w[at] = y[torch.from_numpy(live)]
        for o, w in zip(out, want):
            assert torch.equal(o.cpu(), w)
    assert c.device_status() == 0
    bad = slots.copy()
    bad[rows // 2], bad[3] = pages * page, -9
    c.write(k, v, i32(bad), *scales)
    assert c.device_status() == fp.FP_ERR_DEVICE_BOUNDS
    c.reset_status()
    c.read(i32(bad), *out, k_scale=scales[0], v_scale=scales[1], out_slots=i32(np.arange(rows)))
    assert c.device_status() == fp.FP_ERR_DEVICE_BOUNDS
    assert np.array_equal(c.data.cpu().numpy(), data)        # the same rows where they were, nothing elsewhere


def test_read_to_e4m3_divides_by_the_scale(fp):
    """Scales from 2^-100 to 2^100, negative, zero, infinite and NaN: the quotient is
    fp32's, rounded to e4m3 and saturated, in both read kernels."""
    import torch
    rng = np.random.default_rng(8)
    rows, page, group = 2 ** 11, 64, 64
    scales = np.array([0.0137, 2.0 ** -8, -0.05, 1e-3, 2.0 ** -70, 2.0 ** 70, 0.0, np.inf, np.nan, 3.1e-39], np.float32)
    h = len(scales)
    x = torch.from_numpy(rng.normal(size=(rows, h, 128)).astype(np.float32) * np.where(np.abs(scales) < 1e-3, 1e-3, 1)[:, None])
    x = x.to(torch.bfloat16)
    c = fp.QCache.empty(rows // page, page, h, group)
    slots = i32(np.arange(rows))
    c.write(x.cuda(), x.cuda(), slots)
    values = torch.from_numpy(oq.read(c.data.cpu().numpy(), page, group, np.arange(rows))[0]).float()
    s = torch.from_numpy(scales)
    q = values / s.view(-1, 1)
    want = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for n in (rows, 40):
        out = [torch.zeros((n, h, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
        c.read(slots[:n].contiguous(), *out, k_scale=s.cuda(), v_scale=s.cuda())
        for o in out:
            o = o.cpu()
            nan = torch.isnan(q[:n])
            assert ((o[nan] & 0x7f) == 0x7f).all()
            assert torch.equal(o[~nan], want[:n][~nan])


def test_many_rows_of_special_values(fp):
    """NaN, infinities, constants, ranges below the f16 steps and beyond fp16, in the 16-row kernels."""
    import torch
    rng = np.random.default_rng(3)
    rows = 16400
    x = rng.normal(size=(rows, 1, 128)).astype(np.float32) * 10.0 ** rng.integers(-9, 7, (rows, 1, 1))
    x += 10.0 ** rng.integers(-3, 4, (rows, 1, 1)) * rng.integers(-1, 2, (rows, 1, 1))
    x[::7, 0, 5] = np.nan
    x[::11, 0, 40] = np.inf
    x[::13, 0, 100] = -np.inf
    x[::17] = 2.5
    x = torch.from_numpy(x).to(torch.bfloat16)
    slots = np.arange(rows)
    for group in (32, 64, 128):
        data = np.zeros((-(-rows // 64), 1, 4, oq.chunk_bytes(group)), np.uint8)
        c = fp.QCache(torch.from_numpy(data).cuda(), 64, group)
        c.write(x.cuda(), x.cuda(), i32(slots))
        oq.write(data, 64, group, slots, x.float().numpy(), x.float().numpy())
        got = c.data.cpu().numpy()
        for a, b in zip(oq.read(got, 64, group, slots), oq.read(data, 64, group, slots)):
            assert np.array_equal(a, b, equal_nan=True)
        k, v = c.read(i32(slots))
        want = torch.from_numpy(oq.read(data, 64, group, slots)[0]).float().bfloat16()
        assert torch.equal(torch.nan_to_num(k.cpu().float(), 7.0), torch.nan_to_num(want.float(), 7.0))


def test_write_of_special_values(fp):
    import torch
    x = torch.randn((4, 1, 128))
    x[0, 0, 3], x[0, 0, 40], x[0, 0, 41] = float("nan"), float("inf"), -float("inf")
    x[1, 0, :64] = 2.5                                      # constant groups
    x[1, 0, 64:] = 0.0
    x[2, 0, :32] *= 1e-8                                    # below the f16 steps
    x[2, 0, 32:64] *= 1e30
    x[3, 0, 5] = 3e38
    x = x.to(torch.bfloat16)
    c = fp.QCache(torch.zeros((1, 1, 1, oq.chunk_bytes(32)), dtype=torch.uint8, device="cuda"), 16, 32)
    c.write(x.cuda(), x.cuda(), i32([0, 7, 15, 8]))
    data = np.zeros((1, 1, 1, oq.chunk_bytes(32)), np.uint8)
    oq.write(data, 16, 32, [0, 7, 15, 8], x.float().numpy(), x.float().numpy())
    for got, want in zip(oq.read(c.data.cpu().numpy(), 16, 32, [0, 7, 15, 8]), oq.read(data, 16, 32, [0, 7, 15, 8])):
        assert np.array_equal(got, want, equal_nan=True)
    k, v = c.read(i32([0, 7, 15, 8]))
    assert torch.isnan(k[0, 0, :32]).all() and torch.isfinite(k[0, 0, 32:].float()).all()
    assert c.device_status() == 0


def test_bad_slots_are_skipped_and_reported(fp):
    import torch
    c = fp.QCache(torch.zeros((2, 1, 1, oq.chunk_bytes(64)), dtype=torch.uint8, device="cuda"), 16, 64)
    x, x32, _ = source(1, 4, 1, "bf16")
    c.write(x, x, i32([3, 32, -2, 9]))
    data = np.zeros((2, 1, 1, oq.chunk_bytes(64)), np.uint8)
    oq.write(data, 16, 64, [3, -1, -1, 9], x32, x32)
    assert np.array_equal(c.data.cpu().numpy(), data)
    assert c.device_status() == fp.FP_ERR_DEVICE_BOUNDS
    c.reset_status()
    assert c.device_status() == 0
    k, v = torch.full((3, 1, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 1, 128), dtype=torch.bfloat16,
                                                                                      device="cuda")
    c.read(i32([3, 99, 9]), k, v, out_slots=i32([2, 1, 3]))
    assert c.device_status() == fp.FP_ERR_DEVICE_BOUNDS
    assert (k[:2] == 5).all() and torch.equal(k[2].cpu().float(),
                                              torch.from_numpy(oq.read(data, 16, 64, [3])[0][0]).float().bfloat16().float())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,h,page,mapped", [(1, 1, 16, False), (77, 3, 64, True), (50, 8, 128, False)])
def test_read_rounds_once(fp, rows, h, page, mapped, group, dtype):
    """s * c + m is exact in float64 and rounds once to fp32 in the kernel, then
    to bf16 (or, over the head's scale, to e4m3): bit for bit."""
    import torch
    rng = np.random.default_rng(rows + group)
    pages = 3
    data = np.zeros((pages, h, page // 16, oq.chunk_bytes(group)), np.uint8)
    n = min(rows, pages * page)
    slots = some_slots(9, n, pages * page)
    x, v = rng.normal(size=(2, n, h, 128)).astype(np.float32)
    oq.write(data, page, group, slots, x + 1, v)
    slots[rng.permutation(n)[:n // 5]] = -1
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    to = some_slots(4, n, n + 9) if mapped else np.arange(n)
    shape = (n + 9 if mapped else n, h, 128)
    ks = vs = None
    if dtype == "bf16":
        out = [torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    else:
        ks, vs = (torch.from_numpy((0.005 + 0.02 * rng.random(h)).astype(np.float32)).cuda() for _ in range(2))
        out = [torch.full(shape, 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [o.cpu().clone() for o in out]
    c.read(i32(slots), *out, out_slots=i32(to) if mapped else None, k_scale=ks, v_scale=vs)
    for w, val, s in zip(want, oq.read(data, page, group, slots), (ks, vs)):
        y = torch.from_numpy(val).float()
        y = y.bfloat16() if s is None else (y / s.cpu().view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        live = slots >= 0
        w[torch.from_numpy(to[live])] = y[torch.from_numpy(live)]
    for o, w in zip(out, want):
        assert torch.equal(o.cpu(), w)
    assert c.device_status() == 0


# -- attention ------------------------------------------------------------------------

def attn_case(seed, lens, lq, h_q, h, page, group, dtype="bf16", extra_pages=2, v_scale=1.0, q_scale=1.0, poison=True):
    """A cache with random contents (NaN steps and minima behind the last tokens), queries and tables."""
    import torch
    rng = np.random.default_rng(seed)
    count = [-(-max(0, n) // page) for n in lens]
    pages = sum(count) + extra_pages
    order = rng.permutation(pages)
    table = np.full((len(lens), max(1, max(count))), 10 ** 6, np.int64)
    data = np.zeros((pages, h, page // 16, oq.chunk_bytes(group)), np.uint8)
    n = 128 // group
    # random codes, steps and minima through the byte layout of a chunk
    data[..., :2048] = rng.integers(0, 256, data[..., :2048].shape, dtype=np.uint8)
    half = data[..., 2048:].view(np.float16)                     # [..., 4 * 16 * n]
    step = (0.05 + 0.25 * rng.random(half.shape)).astype(np.float16)
    step[..., 32 * n:48 * n] *= np.float16(v_scale)
    half[...] = step
    m = (rng.normal(size=half.shape) * 0.3 - 1.5).astype(np.float16)
    half[..., 16 * n:32 * n] = m[..., 16 * n:32 * n]
    half[..., 48 * n:] = (m[..., 48 * n:] * np.float16(v_scale)).astype(np.float16)
    at = 0
    for r, c in enumerate(count):
        table[r, :c] = order[at:at + c]
        at += c
    if poison:
        for r, length in enumerate(lens):
            for t in range(max(0, length), count[r] * page):
                _, _, *places = oq._places(t % 16, group)
                chunk = data[table[r, t // page], :, t % page // 16]
                for p in places:
                    for b in p:
                        chunk[:, b:b + 2] = [0, 0x7e]
    total = int(sum(lq))
    q = torch.from_numpy(rng.normal(size=(total, h_q, 128)).astype(np.float32) * q_scale)
    if dtype == "bf16":
        q = q.to(torch.bfloat16)
        return data, table, q.cuda(), q.float().numpy(), None
    s = torch.from_numpy((0.01 + 0.01 * rng.random(h_q)).astype(np.float32)) * q_scale
    c = (q / s.view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return data, table, c.view(torch.uint8).cuda(), (c.float() * s.view(-1, 1)).numpy(), s.cuda()


UNIT_BOUNDS = (0.8, 6.0, 0.8, 6.0)       # steps and minima of groups drawn from N(0, 1)


def tolerances(q32, data, group, ref_o, ref_lse, scale, bounds=None):
    """Output: bf16 rounding of the result (2^-8 of it); two f16 roundings of each
    weight times step (2^-10 of at most 15 steps) and one of each weight times
    minimum (2^-11), both in sums that the weights' total divides; a logit error
    d moves every weight by at most 2 d.  Logits: fp32 sums whose terms' magnitudes
    add up to at most B = scale * sum |q| (15 s + |m|), with fewer than 32 roundings
    of 2^-23 each (2^-18 B), and the exponential's 2^-21."""
    n = 128 // group
    if bounds is None:
        half = np.ascontiguousarray(data[..., 2048:]).view(np.float16).astype(np.float64)
        bounds = (np.nan_to_num(np.abs(half[..., i * 16 * n:(i + 1) * 16 * n])).max() for i in range(4))
    ks, km, vs, vm = bounds
    d = 2.0 ** -18 * scale * np.abs(q32).sum(-1).max() * (15 * ks + km) + 2.0 ** -20
    tol_o = 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -10 * 15 * vs + 2.0 ** -11 * vm + 2 * d * (15 * vs + vm)
    return tol_o, d + 2.0 ** -22 * np.abs(np.nan_to_num(ref_lse, neginf=0.0))


def check_attn(fp, case, lens, lq, page, group, ragged, scale=None, max_q=None):
    import torch
    data, table, q, q32, qs = case
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    cu = i32(np.concatenate([[0], np.cumsum(lq)])) if ragged else None
    out, lse = c.attn(q, i32(table), i32(lens), cu_seqlens_q=cu, max_q=max_q if max_q else max(1, max(lq)), q_scale=qs,
                      softmax_scale=scale or 0.0)
    # a table that has room for long caches has its items cut between thread blocks, a narrow one may not
    wide = np.full((len(lens), max(table.shape[1], 1 + 1024 // page)), 10 ** 6)
    wide[:, :table.shape[1]] = table
    cut, cut_lse = c.attn(q, i32(wide), i32(lens), cu_seqlens_q=cu, max_q=max_q if max_q else max(1, max(lq)), q_scale=qs,
                          softmax_scale=scale or 0.0)
    ref_o, ref_lse = oq.attention(q32, data, page, group, table, lens, lq, scale)
    tol_o, tol_lse = tolerances(q32, data, group, ref_o, ref_lse, scale or 128 ** -0.5)
    assert c.device_status() == 0
    for o, l in ((out, lse), (cut, cut_lse)):
        got, got_lse = o.float().cpu().numpy(), l.cpu().numpy()
        assert np.isfinite(got).all()
        assert np.all(np.abs(got - ref_o) <= tol_o), float((np.abs(got - ref_o) / tol_o).max())
        empty = np.isneginf(ref_lse)
        assert np.array_equal(empty, np.isneginf(got_lse))
        assert np.all(np.abs(got_lse[~empty] - ref_lse[~empty]) <= tol_lse[~empty])
        assert np.all(got.transpose(1, 0, 2)[empty] == 0)
    return out, lse


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,h_q,h,page", [
    ([1], 1, 1, 16), ([2, 0, 15, 16, 17], 4, 1, 16), ([700], 16, 2, 64), ([33, 129, 1, 0, 64, 300], 6, 2, 32),
    ([257, 256, 255], 15, 3, 256), ([1000, 31], 40, 2, 128), ([400, 385, 100], 6, 2, 384)])
def test_decode(fp, lens, h_q, h, page, group, dtype):
    lq = [1] * len(lens)
    check_attn(fp, attn_case(len(lens) + h_q, lens, lq, h_q, h, page, group, dtype), lens, lq, page, group, False)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("lens,lq,h_q,h,page", [
    ([5, 100, 64], [5, 3, 8], 8, 2, 16),              # a prompt from its first token, and drafts
    ([300, 0, 17, 90], [4, 0, 1, 7], 12, 1, 64),      # a request without rows
    ([40, 200], [33, 20], 5, 1, 32),                  # odd chunks
    ([3, 2, 130], [5, 2, 4], 4, 2, 16),               # more queries than tokens: rows without keys
    ([0, 50], [6, 1], 16, 1, 16)])                    # an empty cache with rows
def test_ragged_queries(fp, lens, lq, h_q, h, page, group):
    case = attn_case(sum(lq), lens, lq, h_q, h, page, group)
    a = check_attn(fp, case, lens, lq, page, group, True)
    b = check_attn(fp, case, lens, lq, page, group, True, max_q=1)       # a bound that is too small picks another tile
    assert (a[0].float() - b[0].float()).abs().max() <= 2 ** -6


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("lq,h_q,h", [(2, 16, 2), (3, 16, 2), (5, 16, 2), (8, 16, 2), (1, 32, 2), (1, 12, 1), (4, 20, 4)])
def test_uniform_runs_of_queries(fp, lq, h_q, h, group):
    """Every number of column octets: 16, 24, 40, 64, 16, 12 and 20 columns a kv head."""
    lens = [70, 400, lq]
    case = attn_case(lq, lens, [lq] * 3, h_q, h, 64, group)
    check_attn(fp, case, lens, [lq] * 3, 64, group, False)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("lens,lq", [
    ([90, 300, 5, 1, 0, 64, 33, 200], [1, 9, 1, 1, 1, 1, 1, 1]),     # 8 columns a request in the mean: 36 in tiles of 8
    ([500, 77, 3, 161], [1, 12, 3, 5]),                              # 21: 48 in tiles of 16
    ([40, 610, 6], [6, 6, 6])])                                      # rows that do not differ: 24 in a tile of 32
def test_tiles_by_what_most_requests_fill(fp, lens, lq, group, dtype):
    case = attn_case(31 + sum(lq), lens, lq, 8, 2, 32, group, dtype)
    check_attn(fp, case, lens, lq, 32, group, True)


def test_more_requests_than_a_block_scans_at_once(fp):
    """Ragged rows of 300 requests, some without rows and some without tokens, and the blocks' cuts among them."""
    rng = np.random.default_rng(21)
    lens = rng.integers(0, 60, 300)
    lq = np.minimum(rng.integers(0, 4, 300), np.maximum(lens, 1))
    lens[::17] = 0
    case = attn_case(21, list(lens), list(lq), 6, 2, 16, 64)
    check_attn(fp, case, list(lens), list(lq), 16, 64, True)


@pytest.mark.parametrize("batch,length", [(1, 20000), (3, 5000), (150, 40)])
def test_long_axis_and_many_requests(fp, batch, length):
    rng = np.random.default_rng(batch)
    lens = [length] + list(rng.integers(0, length, batch - 1))
    check_attn(fp, attn_case(batch, lens, [1] * batch, 4, 2, 64, 32), lens, [1] * batch, 64, 32, False)


@pytest.mark.parametrize("q_scale,v_scale", [(30.0, 1.0), (1e-20, 1.0), (1.0, 1e-3), (1.0, 900.0), (2e4, 0.01)])
def test_far_from_unit_scale(fp, q_scale, v_scale):
    """Sharp rows, flat rows, small and large values."""
    lens, lq = [333, 64, 1], [1, 1, 1]
    case = attn_case(5, lens, lq, 8, 2, 64, 32, q_scale=q_scale, v_scale=v_scale)
    check_attn(fp, case, lens, lq, 64, 32, False, scale=0.05)


def test_rising_logits(fp):
    """The running maximum rises at every chunk of a long row."""
    import torch
    L, page = 600, 64
    data, table, q, q32, _ = attn_case(8, [L], [1], 4, 1, page, 32, poison=False)
    unit = q32[0, 0] / np.linalg.norm(q32[0, 0])
    k = np.outer(np.arange(L) / 12.0, unit).astype(np.float32)[:, None]
    t = np.arange(L)
    slots = table[0, t // page] * page + t % page
    oq.write(data, page, 32, slots, k, np.random.default_rng(1).normal(size=(L, 1, 128)).astype(np.float32))
    check_attn(fp, (data, table, q, q32, None), [L], [1], page, 32, False)


def test_q_strides_and_rows_behind_the_last_request(fp):
    import torch
    lens, lq = [90, 200, 7], [2, 1, 3]
    data, table, q, q32, _ = attn_case(3, lens, lq, 8, 2, 16, 64)
    c = fp.QCache(torch.from_numpy(data).cuda(), 16, 64)
    wide = torch.full((9, 14, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:6, 3:11] = q
    out = torch.full((9, 8, 128), 4.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 9), 4.0, device="cuda")
    cu = i32([0, 2, 3, 6])
    c.attn(wide[:, 3:11], i32(table), i32(lens), cu_seqlens_q=cu, max_q=3, out=out, lse=lse)
    a, b = c.attn(q, i32(table), i32(lens), cu_seqlens_q=cu, max_q=3)
    assert torch.equal(out[:6], a) and torch.equal(lse[:, :6], b)
    assert (out[6:] == 4).all() and (lse[:, 6:] == 4).all()
    out2, none = c.attn(q, i32(table), i32(lens), cu_seqlens_q=cu, max_q=3, want_lse=False)
    assert none is None and torch.equal(out2, a)


@pytest.mark.parametrize("width", [0, 80])
def test_bad_device_data_is_reported(fp, width):
    """Page ids out of range read as zeros, lengths out of range as an empty
    cache, rows outside q are left out.  Another length moves the cuts between
    the thread blocks, and with them the rounding of every request: the results
    are held to the oracle, not to the bits of the good call."""
    import torch
    lens, lq = [90, 200, 40], [1, 1, 1]
    data, table, q, q32, _ = attn_case(4, lens, lq, 8, 2, 16, 32)
    if width > table.shape[1]:
        table = np.concatenate([table, np.full((3, width - table.shape[1]), 10 ** 6)], 1)
    c = fp.QCache(torch.from_numpy(data).cuda(), 16, 32)

    def check(out, lse, table, lens, rows=3):
        assert c.device_status() == fp.FP_ERR_DEVICE_BOUNDS
        c.reset_status()
        ref_o, ref_lse = oq.attention(q32, data, 16, 32, table, lens, lq)
        tol_o, tol_lse = tolerances(q32, data, 32, ref_o, ref_lse, 128 ** -0.5)
        assert np.all((np.abs(out.float().cpu().numpy() - ref_o[:rows]) <= tol_o[:rows]))
        ref_lse, tol_lse, got = ref_lse[:, :rows], tol_lse[:, :rows], lse.cpu().numpy()
        live = np.isfinite(ref_lse)
        assert np.all(np.abs(got[live] - ref_lse[live]) <= tol_lse[live]) and np.isneginf(got[~live]).all()

    c.attn(q, i32(table), i32(lens))
    assert c.device_status() == 0
    for value in (-1, data.shape[0], 2 ** 31 - 1):
        bad = table.copy()
        bad[1, 3] = value
        check(*c.attn(q, i32(bad), i32(lens)), bad, lens)
    for value in (-3, table.shape[1] * 16 + 1, 2 ** 31 - 1):             # (a narrow table is not cut, a wide one is)
        out, lse = c.attn(q, i32(table), i32([90, value, 40]))
        assert (out[1] == 0).all()
        check(out, lse, table, [90, 0, 40])
    check(*c.attn(q[:2], i32(table), i32(lens), cu_seqlens_q=i32([0, 1, 2, 3]), max_q=1), table, lens, rows=2)
    # offsets that are no offsets: rows they do not name stay as they were
    out = torch.full((3, 8, 128), 4.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([-5, 1, 2, 3], [0, 2 ** 31 - 1, -2 ** 31, 3], [5, 4, 3, 2], [7, 9, 2 ** 31 - 1, 3]):
        c.attn(q, i32(table), i32(lens), cu_seqlens_q=i32(cu), max_q=1, out=out)
        torch.cuda.synchronize()
    assert c.device_status() == fp.FP_ERR_DEVICE_BOUNDS


def test_repeated_calls_are_bit_identical(fp):
    lens = [3000, 1, 517, 2048]
    data, table, q, q32, _ = attn_case(6, lens, [1] * 4, 32, 4, 64, 32)
    import torch
    c = fp.QCache(torch.from_numpy(data).cuda(), 64, 32)
    first, l1 = c.attn(q, i32(table), i32(lens))
    for _ in range(5):
        again, l2 = c.attn(q, i32(table), i32(lens))
        assert torch.equal(first, again) and torch.equal(l1, l2)


def test_pages_shared_by_requests(fp):
    """Two requests with a common prefix point at the same pages."""
    lens, lq = [150, 140, 64], [1, 1, 1]
    data, table, q, q32, _ = attn_case(31, lens, lq, 8, 2, 32, 32, poison=False)
    table[1, :3] = table[0, :3]
    table[2, :2] = table[0, :2]
    check_attn(fp, (data, table, q, q32, None), lens, lq, 32, 32, False)


def test_offsets_past_32_bits(fp):
    """A cache of 4.7 GB: chunks behind 2^32 bytes are written, read and attended."""
    import torch
    page, h, group, pages = 128, 8, 64, 2 ** 32 // (8 * 8 * 2304) + 3000
    c = fp.QCache.empty(pages, page, h, group)
    assert c.data.numel() > 2 ** 32 + 3000 * 8 * 8 * 2304 - 2 ** 20
    rng = np.random.default_rng(5)
    mine = np.array([pages - 1, 3, pages - 700, pages - 2])
    lens, lq, rows = [350, 100], [1, 1], 450
    table = np.array([[mine[0], mine[1], mine[2]], [mine[3], 0, 0]])
    t = np.arange(350)
    slots = np.concatenate([table[0, t // page] * page + t % page, mine[3] * page + np.arange(100)])
    k, k32, _ = source(1, rows, h, "bf16")
    v, v32, _ = source(2, rows, h, "bf16")
    for part in (slice(0, 449), slice(449, 450)):
        c.write(k[part], v[part], i32(slots[part]))
    # the oracle's cache has just these pages
    small = np.zeros((4, h, page // 16, oq.chunk_bytes(group)), np.uint8)
    to_small = {int(p): i for i, p in enumerate(mine)}
    small_slots = [to_small[int(s) // page] * page + int(s) % page for s in slots]
    oq.write(small, page, group, small_slots, k32, v32)
    for i, p in enumerate(mine):
        n = [128, 128, 94, 100][i]
        rows_i = np.arange(n) + i * page
        for a, b in zip(oq.read(c.data[int(p):int(p) + 1].cpu().numpy(), page, group, np.arange(n)),
                        oq.read(small, page, group, rows_i)):
            assert np.array_equal(a, b)
    back = c.read(i32(slots))
    for got, want in zip(back, oq.read(small, page, group, small_slots)):
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().bfloat16())
    q, q32, _ = source(3, 2, 16, "bf16")
    out, lse = c.attn(q, i32(table), i32(lens))
    ref_o, ref_lse = oq.attention(q32, small, page, group, np.array([[0, 1, 2], [3, 0, 0]]), lens, lq)
    tol_o, tol_lse = tolerances(q32, small, group, ref_o, ref_lse, 128 ** -0.5)
    assert np.all(np.abs(out.float().cpu().numpy() - ref_o) <= tol_o)
    assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= tol_lse)
    assert c.device_status() == 0


def test_lengths_at_the_end_of_an_int_are_refused(fp):
    """A table that has room for 2^31 tokens: a length near that is an empty cache, and reported."""
    import torch
    c = fp.QCache.empty(1, 16, 1, 128)
    c.data.zero_()
    table = torch.zeros((1, 2 ** 27), dtype=torch.int32, device="cuda")
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = c.attn(q, table, i32([2 ** 31 - 1]))
    assert (out == 0).all() and torch.isneginf(lse).all() and c.device_status() == fp.FP_ERR_DEVICE_BOUNDS


def test_nan_and_infinity_reach_their_rows_only(fp):
    """A NaN in one key of one head, an infinite value in another's: the rows that
    attend them are NaN in the columns concerned, the others are what they were."""
    import torch
    lens, lq = [100, 60], [2, 1]
    data, table, q, q32, _ = attn_case(17, lens, lq, 4, 2, 16, 64)
    c = fp.QCache(torch.from_numpy(data).cuda(), 16, 64)
    cu = i32([0, 2, 3])
    good, good_lse = c.attn(q, i32(table), i32(lens), cu_seqlens_q=cu, max_q=2)
    k, v = (t.clone() for t in c.read(i32([table[0, 6] * 16 + 3])))      # request 0's last token
    k[0, 0, 5] = float("nan")
    c.write(k, v, i32([table[0, 6] * 16 + 3]))
    out, lse = c.attn(q, i32(table), i32(lens), cu_seqlens_q=cu, max_q=2)
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[:2, 1]).all()
    for rows in ((0, slice(None)), (1, slice(2, 4)), (2, slice(None))):
        assert torch.isfinite(out[rows].float()).all()
        # the untouched token's codes were written anew by the same quantiser: within half a step of 64 dims
        assert (out[rows].float() - good[rows].float()).abs().max() <= 0.2
    assert torch.equal(out[2], good[2]) and torch.equal(out[0], good[0])
    assert c.device_status() == 0


def test_python_checks_its_tensors(fp):
    import torch
    E = fp.FprefillError
    c = fp.QCache.empty(4, 16, 2, 64)
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    s = i32([1, 2, 3])
    scale = torch.ones(2, device="cuda")
    for bad in (lambda: c.write(x.float(), x.float(), s), lambda: c.write(x, x[:2], s), lambda: c.write(x[:, :1], x[:, :1], s),
                lambda: c.write(x, x, s.long()), lambda: c.write(x, x, s[:2]), lambda: c.write(x, x, s.cpu()),
                lambda: c.write(x.cpu(), x.cpu(), s), lambda: c.write(x[..., :64], x[..., :64], s),
                lambda: c.write(x, x.transpose(0, 1).contiguous().transpose(0, 1), s), lambda: c.write(x, x, s, scale, scale),
                lambda: c.write(x.to(torch.uint8), x.to(torch.uint8), s, scale),
                lambda: c.write(x.to(torch.uint8), x.to(torch.uint8), s, scale, scale[:1]),
                lambda: c.read(s, x), lambda: c.read(s, x, x, out_slots=s[:2]), lambda: c.read(s[:2], x, x),
                lambda: c.read(s, out_slots=s), lambda: c.write(x[..., ::2].repeat(1, 1, 2)[..., ::2], x, s)):
        with pytest.raises(E):
            bad()
    table, lens = i32([[0, 1], [2, 3]]), i32([5, 6])
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: c.attn(q[:, :3], table, lens), lambda: c.attn(q, table[:1], lens), lambda: c.attn(q, table.long(), lens),
                lambda: c.attn(q, table, lens.float()), lambda: c.attn(q, table, lens, cu_seqlens_q=i32([0, 1])),
                lambda: c.attn(q.float(), table, lens), lambda: c.attn(q, table, lens, max_q=2),
                lambda: c.attn(q, table, lens, out=q[:1]), lambda: c.attn(q, table, lens, lse=torch.zeros((2, 4), device="cuda")),
                lambda: c.attn(q, table, lens, q_scale=scale), lambda: c.attn(q, table.cpu(), lens),
                lambda: c.attn(q[..., :64], table, lens), lambda: c.attn(q, table.t(), lens), lambda: c.attn(q, table, lens, max_q=0)):
        with pytest.raises(E):
            bad()
    with pytest.raises(E):
        fp.QCache(c.data, 32, 64)
    with pytest.raises(E):
        fp.QCache(c.data, 16, 32)
    p = fp.PageTables(table, 16, 4, 8)
    for bad in (lambda: p.step(lens[:1], lens, s), lambda: p.step(lens, lens.long(), s), lambda: p.step(lens, lens, s.cpu()),
                lambda: p.step(lens, lens, s, i32([0, 1]))):
        with pytest.raises(E):
            bad()
    assert c.device_status() == 0
    # e4m3 as torch's own type is the same as its codes
    f = torch.randn((3, 2, 128), device="cuda").to(torch.float8_e4m3fn)
    c.write(f, f, s, scale, scale)
    a = c.data.clone()
    c.write(f.view(torch.uint8), f.view(torch.uint8), s, scale, scale)
    assert torch.equal(a, c.data)
    # nothing to do
    c.write(x[:0], x[:0], s[:0])
    out, lse = c.attn(q[:0], table, i32([0, 0]), cu_seqlens_q=i32([0, 0, 0]), max_q=1)
    assert out.shape == (0, 4, 128) and lse.shape == (4, 0) and c.device_status() == 0


# -- together -----------------------------------------------------------------------------

def test_prefill_then_decode(fp):
    """Two requests: tables, the prompt into the 4-bit cache, back into bf16 pages
    for the prefill kernels, then decode steps that advance in place -- eagerly
    and as one captured graph -- against the oracle over the same cache."""
    import torch
    h_q, h, page, group, batch, width, pool = 8, 2, 64, 32, 2, 8, 40
    rng = np.random.default_rng(12)
    free = i32(rng.permutation(pool))
    table = i32(np.zeros((batch, width)))
    c = fp.QCache.empty(pool, page, h, group)
    c.data.random_(0, 256)
    prompt = [256, 130]
    total = sum(prompt)
    step = fp.PageTables(table, page, pool, total)
    step.step(i32([0, 0]), i32(prompt), free)
    k, v, q = (torch.from_numpy(rng.normal(size=(total, n, 128)).astype(np.float32)).to(torch.bfloat16).cuda() for n in
               (h, h, h_q))
    c.write(k, v, step.slots)
    # back into the bf16 pages (the same table), and the dense prefill over them
    kc, vc = (torch.zeros((pool, page, h, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(step.slots, kc.flatten(0, 1), vc.flatten(0, 1), out_slots=step.slots)
    layer = fp.Layer(q, kc, vc, table, [0, prompt[0], total], prompt, [0, 0], h_q, h)
    dense, dense_lse = layer.dense_attn()
    att, att_lse = c.attn(q, table, step.seqlens_k, cu_seqlens_q=step.cu_seqlens_q, max_q=max(prompt))
    assert c.device_status() == 0 and step.device_status() == 0 and layer.device_status() == 0
    # the bf16 pages round the keys by 2^-9 of themselves, the bf16 weights of the prefill by 2^-9
    assert (dense.float() - att.float()).abs().max() <= 4e-2
    assert (dense_lse - att_lse).abs().max() <= 2e-2
    data = c.data.cpu().numpy()
    ref_o, ref_lse = oq.attention(q.float().cpu().numpy(), data, page, group, table.cpu().numpy(), prompt, prompt)
    tol_o, tol_lse = tolerances(q.float().cpu().numpy(), data, group, ref_o, ref_lse, 128 ** -0.5, UNIT_BOUNDS)
    assert np.all(np.abs(att.float().cpu().numpy() - ref_o) <= tol_o)
    assert np.all(np.abs(att_lse.cpu().numpy() - ref_lse) <= tol_lse)

    dec = fp.PageTables(table, page, pool, batch)
    dec.seqlens_k.copy_(step.seqlens_k)
    dec.free_head.copy_(step.free_head)
    ones = i32([1, 1])
    k1, v1 = (torch.zeros((batch, h, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q1 = torch.zeros((batch, h_q, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q1), torch.zeros((h_q, batch), device="cuda")

    def decode():
        dec.step(dec.seqlens_k, ones, free, dec.free_head)
        c.write(k1, v1, dec.slots)
        c.attn(q1, table, dec.seqlens_k, out=out, lse=lse)

    graph = None
    for i in range(70):                                  # past the ends of pages
        for x in (k1, v1, q1):
            x.copy_(torch.from_numpy(rng.normal(size=tuple(x.shape)).astype(np.float32)))
        if i == 3:
            lens, head = dec.seqlens_k.clone(), dec.free_head.clone()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                decode()
            assert torch.equal(lens, dec.seqlens_k) and torch.equal(head, dec.free_head)
        if graph is None:
            decode()
        else:
            graph.replay()
        if i in (0, 2, 3, 40, 69):
            lens = [n + i + 1 for n in prompt]
            assert dec.seqlens_k.tolist() == lens
            data = c.data.cpu().numpy()
            q32 = q1.float().cpu().numpy()
            ref_o, ref_lse = oq.attention(q32, data, page, group, table.cpu().numpy(), lens, [1, 1])
            tol_o, tol_lse = tolerances(q32, data, group, ref_o, ref_lse, 128 ** -0.5, UNIT_BOUNDS)
            assert np.all(np.abs(out.float().cpu().numpy() - ref_o) <= tol_o)
            assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= tol_lse)
    used = sum(-(-(n + 70) // page) for n in prompt)
    assert dec.free_head.item() == used
    assert sorted(table[r, j].item() for r, n in enumerate(prompt) for j in range(-(-(n + 70) // page))) == \
        sorted(free[:used].tolist())
    assert c.device_status() == 0 and dec.device_status() == 0


def test_two_streams_and_another_current_stream(fp):
    """Calls of one cache on two streams at once share no scratch."""
    import torch
    lens = [9000, 4000]
    data, table, q, q32, _ = attn_case(9, lens, [1, 1], 16, 2, 64, 32)
    c = fp.QCache(torch.from_numpy(data).cuda(), 64, 32)
    bt, ln = i32(table), i32(lens)
    qs = [q, q * 2]
    want = [c.attn(x, bt, ln)[0].clone() for x in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for s, x in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(c.attn(x, bt, ln)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_of_one_cache_replayed_at_once(fp):
    """Each captured call has its own scratch: two graphs on two streams do not meet in it."""
    import torch
    lens = [9000, 4000]
    data, table, q, q32, _ = attn_case(9, lens, [1, 1], 16, 2, 64, 32)
    c = fp.QCache(torch.from_numpy(data).cuda(), 64, 32)
    bt, ln = i32(table), i32(lens)
    qs = [q, q * 2]
    want = [c.attn(x, bt, ln)[0].clone() for x in qs]
    outs = [torch.zeros_like(x) for x in qs]
    graphs = []
    for x, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                c.attn(x, bt, ln, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = c.attn(qs[0], bt, ln)[0]
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0]) and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_threads_share_a_cache(fp):
    """Calls from two threads, each on a stream of its own."""
    import threading
    import torch
    data, table, q, q32, _ = attn_case(9, [3000, 700], [1, 1], 16, 2, 64, 32)
    c = fp.QCache(torch.from_numpy(data).cuda(), 64, 32)
    bt, ln = i32(table), i32([3000, 700])
    qs = [q, q * 2]
    want = [c.attn(x, bt, ln)[0].clone() for x in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(x, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                if not torch.equal(c.attn(x, bt, ln)[0], w):
                    wrong.append(1)
    threads = [threading.Thread(target=work, args=a) for a in zip(qs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# -- the tables of many tokens, and batches at the default limit of shared memory ---------------

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,old_max,new_max,page,capacity", [
    (64, 3000, 2600, 64, 100003), (1, 0, 90000, 16, 90001), (2000, 60, 80, 32, 120000), (5, 70000, 30000, 384, 160007)])
def test_page_tables_of_many_tokens(fp, batch, old_max, new_max, page, capacity, in_place):
    """More than 77824 tokens, which the kernel takes eight a thread; capacities that are no multiple of 8."""
    table, old, new, free, pool, cap = tables_case(batch + page, batch, old_max, new_max, page)
    check_tables(fp, table, old, new, free, 2, page, pool, max(cap, capacity), in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables_of_many_tokens_refuse_what_they_cannot_serve(fp, in_place):
    table, old, new, free, pool, cap = tables_case(12, 40, 2000, 6000, 32)
    assert cap > 77829 + 8
    check_tables(fp, table, old, new, free[:len(free) // 2], 2, 32, pool, cap, in_place)     # the free list runs out
    check_tables(fp, table, old, new, free, 2, 32, pool, 77829, in_place)                    # the slot map runs out
    check_tables(fp, table[:, :100], old, new, free, 2, 32, pool, cap, in_place)             # the table is too narrow
    bad = new.copy()
    bad[[3, 17]] = -1, 2 ** 31 - 1
    check_tables(fp, table, old, bad, free, 2, 32, pool, cap, in_place)
    bad = free.copy()
    bad[5] = pool
    check_tables(fp, table, old, new, bad, 2, 32, pool, cap, in_place)


def test_page_tables_of_any_batch_in_a_fresh_process(fp):
    """The scan's 16 bytes a request and the kernel's own arrays pass 48 KB together at 3040
    requests.  A process that has had no larger batch takes them all the same."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import test_qcache_gpu as t\n"
            "from block_sparse_long_fp_gb300 import fprefill as fp\n"
            "for batch in (3039, 3040, 3057, 3071, 3100):\n"
            "    for in_place in (False, True):\n"
            "        table, old, new, free, pool, cap = t.tables_case(batch, batch, 5, 3, 16)\n"
            "        for capacity in (cap, 77900):\n"
            "            t.check_tables(fp, table, old, new, free, 2, 16, pool, capacity, in_place)\n")
    path = os.pathsep.join([root, os.path.join(root, "tests")] + [p for p in [os.environ.get("PYTHONPATH")] if p])
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, PYTHONPATH=path), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_on_one_stream_share_a_cache(fp):
    """Both threads on the default stream, where the calls share scratch: batches, rows and columns
    that differ, long enough to be cut."""
    import threading
    import torch
    data, table, q, q32, _ = attn_case(9, [3000, 700], [3, 3], 16, 2, 64, 32)
    c = fp.QCache(torch.from_numpy(data).cuda(), 64, 32)
    bt, ln = i32(table), i32([3000, 700])
    calls = [(q, bt, ln, 3), (q[:2].contiguous(), bt, ln, 1), (q[:1].contiguous(), bt[:1].contiguous(), ln[:1].contiguous(), 1)]
    want = [tuple(t.clone() for t in c.attn(x, b, n, max_q=m)) for x, b, n, m in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(call, w):
        x, b, n, m = call
        for _ in range(200):
            got = c.attn(x, b, n, max_q=m)
            if not all(torch.equal(a, y) for a, y in zip(got, w)):
                wrong.append(m)
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and c.device_status() == 0


# -- what may lie in a value that a row does not attend ------------------------------------------

@pytest.mark.parametrize("value", ["nan", "inf", "nan step", "nan key"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("lens,lq,h_q,h,page", [
    ([100, 60], [3, 2], 4, 2, 16),             # 8 columns
    ([77, 130], [4, 4], 6, 2, 64),             # 16
    ([300, 33], [8, 8], 8, 2, 32),             # 32
    ([90, 16], [40, 16], 4, 2, 16)])           # several tiles, whose keys end chunks apart
def test_values_behind_a_row_do_not_reach_it(fp, lens, lq, h_q, h, page, group, value):
    """NaN and infinite minima, NaN steps in the last tokens' values (drafts that other rows of the
    request come before): the rows that attend them lose the dims of their group, no other row
    loses anything.  In a key: those rows lose everything, and the others nothing."""
    import torch
    data, table, q, q32, _ = attn_case(23 + sum(lq), lens, lq, h_q, h, page, group)
    n, rng = 128 // group, np.random.default_rng(4)
    clean = data.copy()
    hit = []                                   # (request, token, group), of head 0
    for r in range(2):
        for back in sorted({0, 1, lq[r] // 2}):
            t, g = lens[r] - 1 - back, int(rng.integers(0, n))
            _, _, _, km, vs, vm = oq._places(t % 16, group)
            at = (vs if value == "nan step" else km if value == "nan key" else vm)[g]
            data[table[r, t // page], 0, t % page // 16, at:at + 2] = [0, 0x7c if value == "inf" else 0x7e]
            hit.append((r, t, g))
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    cu = i32(np.concatenate([[0], np.cumsum(lq)]))
    wide = np.full((2, max(table.shape[1], 1 + 1024 // page)), 10 ** 6)
    wide[:, :table.shape[1]] = table
    ref_o, ref_lse = oq.attention(q32, clean, page, group, table, lens, lq)
    tol_o, tol_lse = tolerances(q32, clean, group, ref_o, ref_lse, 128 ** -0.5)
    lost = np.zeros(ref_o.shape, bool)
    for r, t, g in hit:
        for i in range(lq[r]):
            if lens[r] - lq[r] + i >= t:
                lost[sum(lq[:r]) + i, :h_q // h, slice(None) if value == "nan key" else slice(g * group, (g + 1) * group)] = True
    assert lost.any() and not lost.all()
    for bt in (table, wide):
        out, lse = c.attn(q, i32(bt), i32(lens), cu_seqlens_q=cu, max_q=max(lq))
        got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
        assert np.array_equal(~np.isfinite(got), lost)
        assert np.all(np.abs(got - ref_o)[~lost] <= tol_o[~lost])
        if value == "nan key":
            assert np.isnan(got_lse[lost[:, :, 0].T]).all()
        live = ~lost[:, :, 0].T if value == "nan key" else np.ones(ref_lse.shape, bool)
        assert np.array_equal(np.isneginf(got_lse[live]), np.isneginf(ref_lse[live]))
        live &= np.isfinite(ref_lse)
        assert np.all(np.abs(got_lse - ref_lse)[live] <= tol_lse[live])
    assert c.device_status() == 0


def test_infinite_values_are_written_as_the_largest_finite(fp):
    """An infinity in a value is held as 65504, and reaches its group's dims as that."""
    import torch
    lens, lq = [100, 60], [2, 1]
    data, table, q, q32, _ = attn_case(18, lens, lq, 4, 2, 16, 64)
    c = fp.QCache(torch.from_numpy(data).cuda(), 16, 64)
    slot = i32([table[0, 6] * 16 + 3])                                   # request 0's last token
    k, v = (t.clone() for t in c.read(slot))
    v[0, 1, 70], v[0, 1, 80] = float("inf"), -float("inf")
    c.write(k, v, slot)
    data = c.data.cpu().numpy()
    assert oq.read(data, 16, 64, slot.tolist())[1][0, 1, 80] == -65504
    out, lse = c.attn(q, i32(table), i32(lens), cu_seqlens_q=i32([0, 2, 3]), max_q=2)
    ref_o, ref_lse = oq.attention(q32, data, 16, 64, table, lens, lq)
    half = np.nan_to_num(np.ascontiguousarray(data[..., 2048:]).view(np.float16).astype(np.float64))
    vs = half[..., 64:96].max()
    assert vs > 4000 and np.abs(ref_o).max() > 1
    tol_o, tol_lse = tolerances(q32, data, 64, ref_o, ref_lse, 128 ** -0.5)
    assert np.all(np.abs(out.float().cpu().numpy() - ref_o) <= tol_o)
    assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= tol_lse)
    assert c.device_status() == 0


# -- steps of very different sizes in one head's groups ------------------------------------------

@pytest.mark.parametrize("rows,h_q", [(1, 1), (1, 12), (2, 12)])          # 8, 16 and 32 columns
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("big", [16.0, 2000.0])
def test_groups_of_small_steps_beside_large_ones(fp, group, big, rows, h_q):
    """A dominant key in each of the first four chunks (a warp's share each) and a tail of weights
    near 2^-21 of theirs, whose values are all that the first group has, at steps near 2^-11;
    elsewhere in the head, beside the dominant keys, steps of `big`.  400 requests over the same
    pages, so that a warp walks most of its share of a request.

    Every term of the first group's sum is positive (minima of zero, no code in the dominant keys), so
    that roundings of its terms are relative to the sum.  Counted: bf16's half step, 2^-8; the weight
    and its product with the step in fp16, half a step 2^-11 each, and as much again for what the
    second rounds below fp16's normal numbers; twice a logit's error (tolerances) in each weight, and
    as much for the shared sum."""
    import torch
    L, page, batch = 4096, 64, 400
    rng = np.random.default_rng(int(big) + group)
    pages = L // page
    table = rng.permutation(pages + 1)[None, :pages]
    q32 = np.repeat(rng.normal(size=(1, 1, 128)), rows * h_q, 1).reshape(rows, h_q, 128)
    q = torch.from_numpy(q32.astype(np.float32)).to(torch.bfloat16)
    q32 = q.float().numpy()
    scale = 1 / 12.0
    x = q32[0, 0].astype(np.float64)
    # keys: multiples of the query, so that scale q.k spreads around -21 ln 2 of the dominant ones' 6
    want = 6 - 21 * np.log(2) + rng.uniform(-0.7, 0.7, L)
    want[:64:16] = 6
    k = (want / (scale * x @ x))[:, None, None] * x
    v = np.zeros((L, 1, 128))
    data = np.zeros((pages + 1, 1, page // 16, oq.chunk_bytes(group)), np.uint8)
    t = np.arange(L)
    slots = table[0, t // page] * page + t % page
    v[:, 0, 0:group] = np.arange(group) % 16 * (2.0 ** -11 * rng.uniform(0.8, 1.2, (L, 1)))
    v[:64:16, 0, :group] = 0
    v[:, 0, group:] = rng.normal(size=(L, 128 - group))
    v[7:64:16, 0, group:2 * group] = np.arange(group) % 16 * big
    oq.write(data, page, group, slots, k.astype(np.float32), v.astype(np.float32))
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    out, lse = c.attn(q.cuda().repeat(batch, 1, 1), i32(np.repeat(table, batch, 0)), i32([L] * batch), max_q=rows,
                      softmax_scale=scale)
    ref_o, ref_lse = oq.attention(q32, data, page, group, table, [L], [rows], scale)
    tol_o, tol_lse = tolerances(q32, data, group, ref_o, ref_lse, scale)
    got = out.float().cpu().numpy().reshape(batch, rows, h_q, 128)
    got_lse = lse.cpu().numpy().reshape(h_q, batch, rows).transpose(1, 0, 2)
    assert np.all(np.abs(got - ref_o) <= tol_o) and np.all(np.abs(got_lse - ref_lse) <= tol_lse)
    d = tol_lse.max()
    small, ref = got[..., :group], ref_o[..., :group]
    assert ref.max() > 2.0 ** -11 * 15 * 2.0 ** -13    # the tail, 2^-11 of all the weights, is what the group has
    assert np.all(np.abs(small - ref) <= ref * (2.0 ** -8 + 4 * 2.0 ** -11 + 4 * d)), \
        float((np.abs(small - ref) / np.maximum(ref, 1e-30)).max())
    assert c.device_status() == 0


@pytest.mark.parametrize("rows,h_q", [(1, 2), (1, 24), (2, 24)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_steps_that_grow_and_fall_along_a_request(fp, group, rows, h_q):
    """Values from 2^-12 to 2^12 of one, each group of dims by a course of its own."""
    import torch
    L, page, h = 700, 64, 2
    data, table, q, q32, _ = attn_case(14, [L], [rows], h_q, h, page, group, poison=False, q_scale=0.3)
    rng = np.random.default_rng(15)
    t = np.arange(L)
    v = rng.normal(size=(L, h, 128)) + 0.5
    for g in range(128 // group):
        course = 12 * np.sin(t / (40 + 25 * g) + 2 * g)
        v[:, 0, g * group:(g + 1) * group] *= 2.0 ** course[:, None]
        v[:, 1, g * group:(g + 1) * group] *= 2.0 ** -course[::-1, None]
    slots = table[0, t // page] * page + t % page
    k = oq.read(data, page, group, slots)[0]
    oq.write(data, page, group, slots, k.astype(np.float32), v.astype(np.float32))
    out, lse = check_attn(fp, (data, table, q, q32, None), [L], [rows], page, group, False)
    # each group by its own steps: a group that others' tolerance would hide
    ref_o, ref_lse = oq.attention(q32, data, page, group, table, [L], [rows])
    got = out.float().cpu().numpy()
    half = np.ascontiguousarray(data[..., 2048:]).view(np.float16).astype(np.float64)
    n = 128 // group
    bounds = [np.abs(half[..., i * 16 * n:(i + 1) * 16 * n]).max() for i in (0, 1)]
    x = oq.read(data, page, group, slots)[1]
    for a in range(h):
        for g in range(n):
            dims, heads = slice(g * group, (g + 1) * group), slice(a * h_q // h, (a + 1) * h_q // h)
            span = np.abs(x[:, a, dims]).max()
            tol = tolerances(q32, data, group, ref_o, ref_lse, 128 ** -0.5, (*bounds, 2 * span / 15, span))[0]
            assert np.all(np.abs(got - ref_o)[:, heads, dims] <= tol[:, heads, dims])


def test_rows_that_the_requests_do_not_share_evenly_are_refused(fp):
    """Without offsets or max_q every request has total_q / batch rows: 7 rows of 3 requests, 2 of 3."""
    import torch
    c = fp.QCache.empty(4, 16, 2, 64)
    c.data.zero_()
    table, lens = i32([[0, 1], [2, 3], [0, 2]]), i32([5, 6, 7])
    q = torch.zeros((7, 4, 128), dtype=torch.bfloat16, device="cuda")
    for x in (q, q[:2]):
        with pytest.raises(fp.FprefillError):
            c.attn(x, table, lens)
    out, lse = c.attn(q[:6], table, lens)
    assert (out == 0).all() and torch.isfinite(lse).all()
    out, lse = c.attn(q, table, lens, max_q=2, out=torch.full_like(q, 3), lse=torch.full((4, 7), 3.0, device="cuda"))
    assert (out[:6] == 0).all() and (out[6] == 3).all() and (lse[:, 6] == 3).all()
    assert c.device_status() == 0


def test_sizes_kept_for_shapes_are_bounded(fp):
    """A cache object remembers the scratch that a shape takes, of some hundreds of shapes."""
    import torch
    c = fp.QCache.empty(1, 16, 1, 128)
    c.data.zero_()
    table, lens, cu = i32([[0]]), i32([9]), i32([0, 1])
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    for max_q in range(1, 1200):
        out, lse = c.attn(q, table, lens, cu_seqlens_q=cu, max_q=max_q)
    assert (out == 0).all() and len(c._scratch_bytes) <= 512 and c.device_status() == 0


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("which", ["steps", "borders"])
def test_quotients_of_every_step(fp, which, group):
    """The 16-row kernel takes 1 / s and (max - min) / 15 by reciprocals and corrections of its own,
    the other divides: both give the definition's codes, steps and minima.  One row whose heads have
    a scale each: for every f16 step s that a positive range can have, values k s and (k + 1/2) s,
    whose codes are ties that the last bit of 1 / s decides; and ranges within two fp32 steps of 15
    times the border between two f16 steps, which the last bit of the quotient decides."""
    import torch
    rng = np.random.default_rng(6)
    if which == "steps":
        s = np.arange(1, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float32)
        s = s[15 * s <= 65504]                           # the values are clamped there
        codes = np.array([16 * k for k in range(16)] + [8 * (2 * k + 1) for k in range(8)] + [0] * 8, np.float32)
        x = np.tile(codes, 4)[None].repeat(len(s), 0)
        x[:, 32:] = rng.permuted(x[:, 32:], axis=1)
        scale = s / 16
    else:
        f16 = np.arange(1, 0x7bff, dtype=np.uint16).view(np.float16).astype(np.float64)
        border = (f16[:-1] + f16[1:]) / 2
        border = rng.choice(border[15 * border < 65500], 20000, replace=False)
        d = (15 * border).astype(np.float32)
        d = (d.view(np.int32) + rng.integers(-2, 3, d.shape)).astype(np.int32).view(np.float32)
        x = rng.integers(0, 16, (len(d), 128)).astype(np.float32) * 16
        x[:, ::32], x[:, 1::32] = 0, 256
        scale = d / 256
    h = len(scale)
    e4m3 = torch.from_numpy(x).to(torch.float8_e4m3fn)
    assert torch.equal(e4m3.float(), torch.from_numpy(x)) and h >= 16384
    x32 = (x * scale[:, None])[None]
    data = np.zeros((1, h, 1, oq.chunk_bytes(group)), np.uint8)
    oq.write(data, 16, group, [9], x32, x32)
    code, step, _ = oq.quantise(x32, group)
    if which == "steps":
        assert np.array_equal(step[0, :, 0].astype(np.float32), s)
    k = e4m3.view(torch.uint8)[None].cuda()
    sc = torch.from_numpy(scale).cuda()
    for part in (h, 10000):                              # the 16-row kernel, then the one for few rows
        for at in range(0, h, part):
            n = min(part, h - at)
            c = fp.QCache(torch.zeros((1, n, 1, oq.chunk_bytes(group)), dtype=torch.uint8, device="cuda"), 16, group)
            kk, ss = k[:, at:at + n].contiguous(), sc[at:at + n].contiguous()
            c.write(kk, kk, i32([9]), ss, ss)
            got = c.data.cpu().numpy()
            assert np.array_equal(got, data[:, at:at + n]), np.nonzero((got != data[:, at:at + n]).any((0, 2, 3)))[0][:5]


@pytest.mark.parametrize("rows,h_q", [(1, 8), (2, 8), (4, 8)])            # tiles of 8, 16 and 32 columns
def test_sums_of_a_long_request_in_one_block(fp, rows, h_q):
    """456 requests of 262144 tokens over the same pages, which leaves each to a block or two, of
    values of zero mean: what the codes add up to is 300 times the output, and the minima take it
    back.  Counted in each element: bf16's half step, 2^-8.  Two roundings of each weight to fp16,
    2^-11, and the logit's error d (tolerances), which is 2 d of a weight: independent of token to
    token, they add as their roots do, and six times that is taken.  Of the sums of codes and of
    minima, 2^-17: 4096 roundings of at most 2^-24 in each of four warps, of sums that grow, are 2^-20.6
    of them in the spread, six times that 2^-18, and a product's own sum of 16, which is cut towards
    zero below the last bit of its largest term and whose codes are subnormal, as much again."""
    import torch
    n, page, group, batch = 262144, 64, 32, 456
    gen = torch.Generator("cuda").manual_seed(rows)
    pages = n // page
    c = fp.QCache.empty(pages, page, 1, group)
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(1, -1)
    slots = (table[0].long().repeat_interleave(page) * page + torch.arange(n, device="cuda") % page).to(torch.int32)
    k, v = (torch.randn((n, 1, 128), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    c.write(k, v, slots)
    q = (torch.randn((rows, h_q, 128), generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    out, lse = c.attn(q.repeat(batch, 1, 1), table.repeat(batch, 1).contiguous(),
                      torch.full((batch,), n, dtype=torch.int32, device="cuda"), max_q=rows)
    data = c.data.cpu().numpy()
    k, v = (torch.from_numpy(x[:, 0]).cuda() for x in oq.read(data, page, group, slots.cpu().numpy()))
    got, got_lse = out.view(batch, rows, h_q, 128).double(), lse.view(h_q, batch, rows).double()
    low = v.view(n, 128 // group, group).amin(-1, keepdim=True).expand(-1, -1, group).reshape(n, 128)
    half = np.ascontiguousarray(data[..., 2048:]).view(np.float16).astype(np.float64)
    ks, km = (np.abs(half[..., x * 64:(x + 1) * 64]).max() for x in (0, 1))
    d = 2.0 ** -18 * 128 ** -0.5 * float(q.double().abs().sum(-1).max()) * (15 * ks + km) + 2.0 ** -20
    for i in range(rows):
        z = (q[i].double() @ k.t()) / 128 ** 0.5
        z[:, n - rows + i + 1:] = -float("inf")
        want_lse = torch.logsumexp(z, -1)
        w = torch.exp(z - want_lse.unsqueeze(-1))
        ref = w @ v
        spread = 2.0 ** -11 * torch.sqrt((w * w) @ ((v - low) ** 2 + v ** 2)) + 2 * d * torch.sqrt((w * w) @ v ** 2)
        tol = 2.0 ** -8 * ref.abs() + 6 * spread + 2.0 ** -17 * (w @ (v - low) + w @ low.abs())
        for r in (0, 1, 200, batch - 1):
            assert ((got[r, i] - ref).abs() <= tol).all(), float(((got[r, i] - ref).abs() / tol).max())
            assert ((got_lse[:, r, i] - want_lse).abs() <= d + 2.0 ** -22 * want_lse.abs()).all()
    assert c.device_status() == 0


def test_tensors_handed_over_between_streams(fp):
    """Rows made on one stream, behind a wait, and written, attended and read on another that an
    event holds back: the launches' early start is for the kernel before them in their own stream."""
    import torch
    lens, h, page, group = [500, 70], 2, 64, 32
    data, table, q, q32, _ = attn_case(41, lens, [1, 1], 8, h, page, group)
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    bt, ln = i32(np.concatenate([table, np.full((2, 20), 10 ** 6)], 1)), i32(lens)
    slot = i32([table[0, 499 // page] * page + 499 % page, table[1, 1] * page + 5])
    rows = [source(50 + i, 2, h, "bf16")[0] for i in range(6)]
    kept = c.data.clone()
    want = []
    for r in rows:
        c.write(r, r, slot)
        want.append((c.attn(q, bt, ln)[0].clone(), c.read(slot)[0].clone()))
    assert not torch.equal(want[0][0], want[1][0])
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    k = torch.zeros_like(rows[0])
    for _ in range(5):
        c.data.copy_(kept)
        torch.cuda.synchronize()
        got = []
        for r in rows:
            with torch.cuda.stream(one):
                one.wait_stream(two)
                torch.cuda._sleep(200000)
                k.copy_(r)
            with torch.cuda.stream(two):
                c.attn(q, bt, ln)                        # something of its own before
                two.wait_stream(one)
                c.write(k, k, slot)
                got.append((c.attn(q, bt, ln)[0], c.read(slot)[0]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert c.device_status() == 0


@pytest.mark.parametrize("rows,h_q", [(2, 2), (4, 6), (8, 6)])
@pytest.mark.parametrize("length", [12, 300])
def test_an_infinite_value_of_a_later_row(fp, length, rows, h_q):
    """An infinity (65504 in the cache, in steps of up to 8734) in the last token's values, which only
    the last row attends.  The rows before it lose what fp16 loses of their own steps beside that one:
    2^-25 of it a step, 15 steps a code, 0.004 of an output's unit at most, and their other roundings."""
    import torch
    lens, lq, h, page, group = [length], [rows], 2, 16, 32
    data, table, q, q32, _ = attn_case(61 + rows, lens, lq, h_q, h, page, group)
    clean = data.copy()
    c = fp.QCache(torch.from_numpy(data).cuda(), page, group)
    slot = i32([table[0, (length - 1) // page] * page + (length - 1) % page])
    k, v = (t.clone() for t in c.read(slot))
    v[0, :, 40], v[0, :, 41], v[0, 1, 100] = float("inf"), -float("inf"), float("inf")
    c.write(k, v, slot)
    data = c.data.cpu().numpy()
    ref_o, ref_lse = oq.attention(q32, data, page, group, table, lens, lq)
    ref_clean, _ = oq.attention(q32, clean, page, group, table, lens, lq)
    assert np.allclose(ref_o[:-1], ref_clean[:-1]) and np.abs(ref_o[-1]).max() > 2
    half = np.ascontiguousarray(clean[..., 2048:]).view(np.float16).astype(np.float64)
    bounds = [np.nan_to_num(np.abs(half[..., i * 64:(i + 1) * 64])).max() for i in range(4)]
    wide = np.full((1, table.shape[1] + 100), 10 ** 6)
    wide[:, :table.shape[1]] = table
    for bt in (table, wide):
        out, lse = c.attn(q, i32(bt), i32(lens), max_q=rows)
        got = out.float().cpu().numpy()
        tol, tol_lse = tolerances(q32, clean, group, ref_o, ref_lse, 128 ** -0.5, bounds)
        assert np.all(np.abs(got - ref_o)[:-1] <= tol[:-1] + 15 * 2.0 ** -25 * 8736)
        tol = tolerances(q32, data, group, ref_o, ref_lse, 128 ** -0.5)[0]
        assert np.all(np.abs(got - ref_o)[-1] <= tol[-1])
        assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= tol_lse)
    assert c.device_status() == 0

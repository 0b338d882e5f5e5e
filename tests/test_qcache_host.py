"""The serving operators without a GPU: argument checks of the C ABI (no call
here reaches a launch), and pins of their float64 oracle."""
import ctypes

import numpy as np
import pytest

from oracle import qcache as oq

P = 4096                                  # a non-null, aligned address that nothing reads


@pytest.fixture(scope="module")
def fp():
    from block_sparse_long_fp_gb300 import build, fprefill
    build.build()
    return fprefill


def cache(fp, **over):
    c = fp.FpQCache(P, 10, 64, 4, 128, 32)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def tables(fp, **over):
    t = fp.FpTables(4, 64, 100, 8, 50, 32, *[P] * 10)
    for k, v in over.items():
        setattr(t, k, v)
    return t


def rows(fp, **over):
    r = fp.FpQCacheRows(5, fp.FP_BF16, P, P, 512, 128, P, 0, 5, 0, 0)
    for k, v in over.items():
        setattr(r, k, v)
    return r


def query(fp, **over):
    q = fp.FpQCacheQuery(3, 16, 3, 1, fp.FP_BF16, P, 2048, 128, 0, 0, P, P, 8, 0.0)
    for k, v in over.items():
        setattr(q, k, v)
    return q


def test_sizes(fp):
    L = fp.lib()
    for group in (32, 64, 128):
        c = cache(fp, group=group)
        assert L.fp_qcache_chunk_bytes(c) == oq.chunk_bytes(group) == fp.QCache.chunk_bytes(group)
        assert L.fp_qcache_bytes(c) == 10 * 4 * 4 * oq.chunk_bytes(group)
    big = cache(fp, num_pages=(1 << 25) - 1, h_kv=8)        # sizes pass 32 bits
    assert L.fp_qcache_bytes(big) == ((1 << 25) - 1) * 8 * 4 * 2560
    assert L.fp_qcache_attn_scratch_bytes(cache(fp), query(fp)) >= 16
    for bad in (dict(group=16), dict(d=64), dict(page_size=48), dict(page_size=8), dict(num_pages=0), dict(h_kv=0),
                dict(num_pages=1 << 25)):
        assert L.fp_qcache_bytes(cache(fp, **bad)) == 0
        assert L.fp_qcache_attn_scratch_bytes(cache(fp, **bad), query(fp)) == 0


@pytest.mark.parametrize("over,code", [
    (dict(batch=0), 1), (dict(batch=4097), 2), (dict(page_size=48), 2), (dict(num_pages=0), 1),
    (dict(num_pages=1 << 25), 2), (dict(max_pages_per_seq=0), 1), (dict(num_free=-1), 1), (dict(capacity=0), 1),
    (dict(seqlens=None), 1), (dict(new_lens=None), 1), (dict(free_pages=None), 1), (dict(block_table=None), 1),
    (dict(cu_seqlens_q=None), 1), (dict(seqlens_k=None), 1), (dict(positions=None), 1), (dict(slots=None), 1),
    (dict(free_next=None), 1), (dict(positions=P + 4), 1), (dict(slots=P + 8), 1), (dict(seqlens=P + 2), 1),
])
def test_page_tables_refusals(fp, over, code):
    assert fp.lib().fp_page_tables(tables(fp, **over), P, 256, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(dtype=7), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1),
    (dict(k=P + 8), 1), (dict(stride_head=120), 1), (dict(stride_tok=500), 1), (dict(stride_tok=516), 1),
    (dict(stride_head=132, stride_tok=1024), 1), (dict(dtype=1), 1), (dict(dtype=1, k_scale=P), 1),
    (dict(slots=P + 1), 1), (dict(rows=(1 << 30) + 1, out_rows=2 ** 31 - 1), 2),
])
def test_rows_refusals(fp, over, code):
    L = fp.lib()
    assert L.fp_qcache_write(cache(fp), rows(fp, **over), P, 256, None) == code
    assert L.fp_qcache_read(cache(fp), rows(fp, **over), P, 256, None) == code


def test_read_targets_and_caches_are_checked(fp):
    L = fp.lib()
    assert L.fp_qcache_read(cache(fp), rows(fp, out_rows=4), P, 256, None) == fp.FP_ERR_INVALID
    assert L.fp_qcache_read(cache(fp), rows(fp, out_rows=-1, out_slots=P), P, 256, None) == fp.FP_ERR_INVALID
    for bad, code in ((dict(data=None), 1), (dict(data=P + 8), 1), (dict(group=48), 2), (dict(d=64), 2),
                      (dict(page_size=100), 2), (dict(h_kv=0), 1)):
        assert L.fp_qcache_write(cache(fp, **bad), rows(fp), P, 256, None) == code
        assert L.fp_qcache_read(cache(fp, **bad), rows(fp), P, 256, None) == code
        assert L.fp_qcache_attn(cache(fp, **bad), query(fp), P, None, P, 1 << 40, P, 256, None) == code
    # nothing to do is done
    assert L.fp_qcache_write(cache(fp), rows(fp, rows=0, k=None), P, 256, None) == fp.FP_OK
    assert L.fp_qcache_attn(cache(fp), query(fp, total_q=0, q=None, cu_seqlens_q=P), None, None, P, 1 << 40, P, 256,
                            None) == fp.FP_OK


@pytest.mark.parametrize("over,code", [
    (dict(batch=0), 1), (dict(batch=4097), 2), (dict(h_q=18), 1), (dict(h_q=0), 1), (dict(total_q=-1), 1),
    (dict(max_q=0), 1), (dict(max_q=2), 1), (dict(dtype=3), 1), (dict(dtype=1), 1), (dict(q=None), 1),
    (dict(q=P + 8), 1), (dict(q_stride_head=64), 1), (dict(q_stride_tok=2000), 1), (dict(q_stride_tok=2052), 1),
    (dict(seqlens_k=None), 1), (dict(block_table=None), 1), (dict(max_pages_per_seq=0), 1),
    (dict(cu_seqlens_q=P + 2), 1), (dict(total_q=1 << 30, cu_seqlens_q=P), 2),
])
def test_attention_refusals(fp, over, code):
    assert fp.lib().fp_qcache_attn(cache(fp), query(fp, **over), P, None, P, 1 << 40, P, 256, None) == code


def test_scales_that_are_not_aligned_are_refused(fp):
    L = fp.lib()
    for over in (dict(k_scale=P + 2, v_scale=P), dict(k_scale=P, v_scale=P + 1)):
        r = rows(fp, dtype=fp.FP_E4M3, **over)
        assert L.fp_qcache_write(cache(fp), r, P, 256, None) == fp.FP_ERR_INVALID
        assert L.fp_qcache_read(cache(fp), r, P, 256, None) == fp.FP_ERR_INVALID
    q = query(fp, dtype=fp.FP_E4M3, q_scale=P + 2)
    assert L.fp_qcache_attn(cache(fp), q, P, None, P, 1 << 40, P, 256, None) == fp.FP_ERR_INVALID


def test_workspaces_are_checked(fp):
    L = fp.lib()
    for ws, n in ((None, 256), (P, 255)):
        assert L.fp_page_tables(tables(fp), ws, n, None) == fp.FP_ERR_WORKSPACE
        assert L.fp_qcache_write(cache(fp), rows(fp), ws, n, None) == fp.FP_ERR_WORKSPACE
        assert L.fp_qcache_read(cache(fp), rows(fp), ws, n, None) == fp.FP_ERR_WORKSPACE
        assert L.fp_qcache_attn(cache(fp), query(fp), P, None, P, 1 << 40, ws, n, None) == fp.FP_ERR_WORKSPACE
    need = L.fp_qcache_attn_scratch_bytes(cache(fp), query(fp))
    for scratch, n in ((None, need), (P, need - 1), (P + 8, need)):
        assert L.fp_qcache_attn(cache(fp), query(fp), P, None, scratch, n, P, 256, None) == fp.FP_ERR_WORKSPACE
    assert L.fp_qcache_attn(cache(fp), query(fp), None, None, P, need, P, 256, None) == fp.FP_ERR_INVALID


def test_python_refuses_host_tensors(fp):
    import torch
    with pytest.raises(fp.FprefillError):
        fp.QCache(torch.zeros((1, 1, 4, 2560), dtype=torch.uint8), 64)
    with pytest.raises(fp.FprefillError):
        fp.PageTables(torch.zeros((1, 1), dtype=torch.int32), 64, 1, 1)
    with pytest.raises(fp.FprefillError):
        fp.QCache.empty(1, 64, 1, group=48, device="cpu")


def test_one_call_at_a_time_fills_a_streams_scratch(fp):
    """The attention enqueues two kernels that hand partial results over in scratch.  Two threads
    on one stream share it, so that no second call may come between a first one's kernels."""
    import threading
    import time
    import types
    import torch
    c = object.__new__(fp.QCache)
    cuda = types.SimpleNamespace(is_current_stream_capturing=lambda: False)
    busy, met = set(), []

    def entry(*args):                          # stands in for the library: enqueues, waits, enqueues
        scratch = args[-5]
        met.append(scratch in busy)
        busy.add(scratch)
        time.sleep(0.002)
        busy.discard(scratch)
        return fp.FP_OK
    c.__dict__.update(_torch=types.SimpleNamespace(cuda=cuda, empty=torch.empty, uint8=torch.uint8), device="cpu", _index=0,
                      _stream=lambda index: 7, _scratch={}, _lock=threading.Lock(), _f=(None, None, entry), _ws_ptr=P)
    threads = [threading.Thread(target=lambda: [c._attn((b"", b"", P, 0), 1000) for _ in range(20)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(met) == 80 and not any(met)


# -- pins of the oracle ---------------------------------------------------------

@pytest.mark.parametrize("group", [32, 64, 128])
def test_oracle_quantisation_is_within_half_a_step(group):
    x = np.random.default_rng(1).normal(size=(50, 2, 128)).astype(np.float32) * 3 + 1
    code, step, low = oq.quantise(x, group)
    y = oq.values(code, step, low, group)
    s = np.repeat(step.astype(np.float64), group, -1)
    m = np.repeat(np.abs(low.astype(np.float64)), group, -1)
    # half a step; the ends may clip by the rounding of minimum (2^-11) and of 15 steps (2^-11)
    assert np.all(np.abs(y - x) <= s / 2 * (1 + 1e-5) + 2.0 ** -11 * (m + 15 * s))
    assert code.max() == 15 and code.min() == 0


def test_oracle_cache_is_a_bijection_of_tokens():
    """Every byte of a chunk belongs to one token; what is written is read, and only that."""
    rng = np.random.default_rng(2)
    for group in (32, 64, 128):
        seen = np.zeros(oq.chunk_bytes(group) * 2, int)
        for t in range(16):
            k, v, *f16 = oq._places(t, group)
            for b, n in k + v:
                seen[2 * b + n] += 1
            for at in f16:
                for b in at:
                    seen[2 * b:2 * b + 4] += 1
        assert np.all(seen == 1)
        data = rng.integers(0, 256, (3, 2, 2, oq.chunk_bytes(group)), dtype=np.uint8)
        before = data.copy()
        slots = [5, 37, 16, 95]
        k, v = rng.normal(size=(2, 4, 2, 128)).astype(np.float32)
        oq.write(data, 32, group, slots, k, v)
        got = oq.read(data, 32, group, slots)
        for x, y in zip((k, v), got):
            assert np.array_equal(oq.values(*oq.quantise(x, group), group), y)
        others = [s for s in range(96) if s not in slots]
        for x, y in zip(oq.read(before, 32, group, others), oq.read(data, 32, group, others)):
            assert np.array_equal(x, y, equal_nan=True)


def test_oracle_special_values():
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, 3], x[0, 0, 40], x[0, 0, 41], x[0, 0, 70] = np.nan, np.inf, -np.inf, 7.0
    y = oq.values(*oq.quantise(x, 32), 32)[0, 0]
    assert np.isnan(y[:32]).all() and np.isfinite(y[32:]).all()
    assert y[40] > 65000 and y[41] == -65504 and abs(y[70] - 7) < 1e-2 and np.all(y[96:] == 0)


def test_oracle_attention_of_one_and_of_equal_keys():
    rng = np.random.default_rng(3)
    data = np.zeros((4, 1, 1, oq.chunk_bytes(32)), np.uint8)
    v = rng.normal(size=(20, 1, 128)).astype(np.float32)
    k = np.repeat(rng.normal(size=(1, 1, 128)).astype(np.float32), 20, 0)
    table = np.array([[2, 0]])
    oq.write(data, 16, 32, [32 + t if t < 16 else t - 16 for t in range(20)], k, v)
    q = rng.normal(size=(1, 2, 128))
    _, vv = oq.read(data, 16, 32, [32 + t if t < 16 else t - 16 for t in range(20)])
    o, lse = oq.attention(q, data, 16, 32, table, [1], [1])
    assert np.allclose(o[0], vv[0]) and o.shape == (1, 2, 128)
    o, lse20 = oq.attention(q, data, 16, 32, table, [20], [1])
    assert np.allclose(o[0], vv.mean(0)) and np.allclose(lse20 - lse, np.log(20))
    o, lse = oq.attention(q, data, 16, 32, table, [0], [1])
    assert np.all(o == 0) and np.all(lse == -np.inf)

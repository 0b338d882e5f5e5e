"""Rotary positions and the bf16 / e4m3 paged cache without a GPU: argument checks
of the C ABI (no call here reaches a launch), the frequencies, and pins of their
float64 oracle."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from oracle import cache as oc

P = 4096                                  # a non-null, aligned address that nothing reads
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)


@pytest.fixture(scope="module")
def fp():
    from block_sparse_long_fp_gb300 import build, fprefill
    build.build()
    return fprefill


def filled(x, over):
    for k, v in over.items():
        setattr(x, k, v)
    return x


def rope_table(fp, **over):
    return filled(fp.FpRopeTable(128, 0, 1.0, P), over)


def rope_rows(fp, **over):
    return filled(fp.FpRopeRows(5, 4, P, 512, 128, P, 512, 128, fp.FP_BF16, 0, P, 0), over)


def cache(fp, **over):
    return filled(fp.FpCache(P, P, 10, 64, 4, 128, fp.FP_BF16, 0, 0), over)


def rows(fp, **over):
    return filled(fp.FpCacheRows(5, 8, P, P, P, 512, 128, 512, 128, 1024, 128, P, 1024, 128, fp.FP_BF16, 0, P, P), over)


# -- frequencies ----------------------------------------------------------------

def test_turns_are_the_fraction_of_a_turn_to_64_bits(fp):
    rng = np.random.default_rng(0)
    f = np.concatenate([500000.0 ** (-np.arange(64) / 64), 10.0 ** rng.uniform(-12, 6, 200), [0.0, 2.0 ** 20, 2 * np.pi]])
    f = np.concatenate([f, -f])
    got = np.zeros(f.size, np.uint64)
    assert fp.lib().fp_rope_turns(f.ctypes.data, f.size, got.ctypes.data) == 0
    for x, t in zip(f, got):
        want = Fraction(float(x)) / (2 * PI) % 1 * 2 ** 64
        # two quotients of doubles carry 2^-104 of the value: below a unit up to 2^20 / 2 pi = 2^17.3 turns,
        # plus the unit's own rounding
        off = (int(t) - want + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= 1, (x, off)


def test_turns_refusals(fp):
    f, t = np.ones(4), np.zeros(4, np.uint64)
    L = fp.lib()
    assert L.fp_rope_turns(None, 4, t.ctypes.data) == 1
    assert L.fp_rope_turns(f.ctypes.data, 4, None) == 1
    assert L.fp_rope_turns(f.ctypes.data, 0, t.ctypes.data) == 1
    for bad in (np.nan, np.inf, -np.inf, 2.0 ** 20 + 1):
        f[2] = bad
        assert L.fp_rope_turns(f.ctypes.data, 4, t.ctypes.data) == 1


def test_frequencies(fp):
    F = fp.rope_frequencies
    i = np.arange(64)
    plain = F(128, 10000.0)
    assert np.allclose(plain, 10000.0 ** (-i / 64), rtol=1e-14)
    assert np.allclose(F(128, 10000.0, "linear", 4.0), plain / 4, rtol=1e-14)
    raised = F(128, 10000.0, "base", 4.0)
    assert raised[0] == 1 and np.isclose(raised[-1], plain[-1] / 4, rtol=1e-12)
    for kind, kw in (("smooth", dict(low=1.0, high=4.0)), ("ramp", dict(low=1.0, high=32.0))):
        f = F(128, 500000.0, kind, 8.0, original=8192, **kw)
        p = F(128, 500000.0)
        waves = 8192 * p / (2 * np.pi)
        ratio = f / p
        assert np.allclose(ratio[waves > 1.3 * kw["high"]], 1, rtol=1e-12)          # "ramp" rounds its ends outwards,
        assert np.allclose(ratio[waves < 0.7 * kw["low"]], 1 / 8, rtol=1e-12)       # by less than a pair
        assert np.all(np.diff(ratio) <= 1e-12) and ratio.min() >= 0.125 - 1e-12
    assert F(2, 10000.0).tolist() == [1.0] and F(64).size == 32
    for bad in (dict(rot=3), dict(rot=0), dict(rot=130), dict(base=1.0), dict(factor=0.0), dict(scaling="other"),
                dict(scaling="smooth", low=4.0), dict(scaling="ramp", original=0), dict(rot=2, scaling="base")):
        with pytest.raises(fp.FprefillError):
            F(**bad)


# -- refusals ---------------------------------------------------------------------

@pytest.mark.parametrize("over,code", [
    (dict(rot=0), 1), (dict(rot=127), 1), (dict(rot=130), 1), (dict(layout=2), 1), (dict(turns=None), 1),
    (dict(turns=P + 4), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
])
def test_rope_table_refusals(fp, over, code):
    L = fp.lib()
    assert L.fp_rope(rope_table(fp, **over), rope_rows(fp), None) == code
    assert L.fp_cache_append(cache(fp), rope_table(fp, **over), rows(fp), P, 256, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(heads=0), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(positions=None), 1),
    (dict(x=P + 8), 1), (dict(out=P + 8), 1), (dict(positions=P + 2), 1), (dict(x_stride_head=120), 1),
    (dict(x_stride_tok=504), 1), (dict(x_stride_tok=516), 1), (dict(out_stride_tok=504), 1), (dict(out_dtype=5), 1),
    (dict(out_dtype=1), 1), (dict(out_dtype=1, out_scale=P + 2), 1), (dict(out_dtype=1, out_scale=P, out_stride_tok=520), 1),
    (dict(inverse=2), 1), (dict(x_stride_tok=1 << 41), 1), (dict(rows=(1 << 30) + 1), 2),
    (dict(heads=(1 << 16) + 1, x_stride_tok=1 << 30, out_stride_tok=1 << 30), 2), (dict(rows=1 << 29, heads=17), 2),
])
def test_rope_refusals(fp, over, code):
    assert fp.lib().fp_rope(rope_table(fp), rope_rows(fp, **over), None) == code


def test_calls_without_rows_do_nothing(fp):
    L = fp.lib()
    assert L.fp_rope(rope_table(fp), rope_rows(fp, rows=0, x=None, out=None, positions=None), None) == 0
    assert L.fp_cache_append(cache(fp), None, rows(fp, rows=0, k=None, v=None, slots=None), P, 256, None) == 0


@pytest.mark.parametrize("over,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=P + 8), 1), (dict(num_pages=0), 1), (dict(page_size=48), 2),
    (dict(page_size=8), 2), (dict(num_pages=1 << 25), 2), (dict(h_kv=0), 1), (dict(d=64), 2), (dict(dtype=3), 1),
    (dict(dtype=1), 1), (dict(dtype=1, k_scale=P), 1), (dict(dtype=1, k_scale=P, v_scale=P + 2), 1),
])
def test_cache_refusals(fp, over, code):
    assert fp.lib().fp_cache_append(cache(fp, **over), rope_table(fp), rows(fp), P, 256, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(h_q=-1), 1), (dict(h_q=0), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(slots=None), 1), (dict(slots=P + 1), 1), (dict(positions=None), 1), (dict(positions=P + 2), 1),
    (dict(q_out=None), 1), (dict(q_dtype=4), 1), (dict(q_dtype=1), 1), (dict(q_dtype=1, q_scale=P + 2), 1),
    (dict(k_stride_tok=500), 1), (dict(v_stride_head=64), 1), (dict(q_stride_tok=1020), 1), (dict(q_out_stride_tok=1020), 1),
    (dict(k=P + 2), 1), (dict(v=P + 8), 1), (dict(q=P + 4), 1), (dict(rows=(1 << 30) + 1), 2), (dict(rows=1 << 30), 2),
])
def test_append_refusals(fp, over, code):
    assert fp.lib().fp_cache_append(cache(fp), rope_table(fp), rows(fp, **over), P, 256, None) == code


def test_workspace_is_wanted(fp):
    L = fp.lib()
    assert L.fp_cache_append(cache(fp), None, rows(fp), None, 256, None) == 3
    assert L.fp_cache_append(cache(fp), None, rows(fp), P, 255, None) == 3
    assert L.fp_cache_append(cache(fp), None, rows(fp), P + 2, 256, None) == 1
    assert L.fp_cache_append(None, None, rows(fp), P, 256, None) == 1
    assert L.fp_cache_append(cache(fp), None, None, P, 256, None) == 1
    assert L.fp_rope(None, rope_rows(fp), None) == 1 and L.fp_rope(rope_table(fp), None, None) == 1


# -- pins of the oracle -------------------------------------------------------------

def test_oracle_codes():
    v = oc.e4m3_values(np.arange(256))
    assert v[0x7e] == 448 and v[0x38] == 1 and v[1] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and np.isnan(v[[0x7f, 0xff]]).all()
    assert np.array_equal(v[128:255], -v[:127])


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_a_rotation(interleaved):
    """Scores depend on the distance alone, the inverse undoes it, dims behind it stay."""
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(24) / 24)
    q, k = rng.normal(size=(2, 1, 3, 128))
    a = oc.rope(q, [70], f, interleaved) * oc.rope(k, [50], f, interleaved)
    b = oc.rope(q, [1020], f, interleaved) * oc.rope(k, [1000], f, interleaved)
    assert np.allclose(a.sum(-1), b.sum(-1), atol=1e-11)
    r = oc.rope(q, [12345], f, interleaved, 1.5)
    assert np.array_equal(r[..., 48:], q[..., 48:])
    assert np.allclose(oc.rope(r, [12345], f, interleaved, 1 / 1.5, inverse=True), q, atol=1e-12)
    e = np.zeros((1, 1, 128))
    e[0, 0, 2 if interleaved else 1] = 1                        # pair 1 at position 3
    y = oc.rope(e, [3], f, interleaved)[0, 0]
    assert np.isclose(y[2 if interleaved else 1], np.cos(3 * f[1])) and np.isclose(y[3 if interleaved else 25], np.sin(3 * f[1]))


def test_oracle_attention_is_softmax_attention():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(2, 4, 16, 2, 128))
    table = np.array([[2, 0, 3]])
    q = rng.normal(size=(3, 4, 128))
    o, lse = oc.attention(q, k, v, table, [35], [3])
    kr, vr = (x[[2, 0, 3]].reshape(48, 2, 128) for x in (k, v))
    for i in range(3):
        for a in range(4):
            z = kr[:33 + i, a // 2] @ q[i, a] / np.sqrt(128)
            p = np.exp(z)
            assert np.allclose(o[i, a], p @ vr[:33 + i, a // 2] / p.sum()) and np.isclose(lse[a, i], np.log(p.sum()))
    o, lse = oc.attention(q, k, v, table, [2], [3])              # the first row has no key
    assert not o[0].any() and np.all(lse[:, 0] == -np.inf) and np.all(np.isfinite(lse[:, 1:]))


# -- the attention's refusals -------------------------------------------------------

def query(fp, **over):
    return filled(fp.FpQCacheQuery(3, 16, 3, 1, fp.FP_BF16, P, 2048, 128, 0, 0, P, P, 8, 0.0), over)


def attn(fp, c=None, q=None, out=P, lse=P, scratch=P, scratch_bytes=1 << 40, ws=P, ws_bytes=256):
    return fp.lib().fp_cache_attn(c or cache(fp), q or query(fp), out, lse, scratch, scratch_bytes, ws, ws_bytes, None)


@pytest.mark.parametrize("over,code", [
    (dict(batch=0), 1), (dict(batch=4097, total_q=5000), 2), (dict(h_q=6), 1), (dict(h_q=0), 1), (dict(total_q=-1), 1),
    (dict(max_q=0), 1), (dict(max_q=2), 1), (dict(dtype=5), 1), (dict(q=None), 1), (dict(q=P + 8), 1),
    (dict(q_stride_tok=2040), 1), (dict(q_stride_head=64), 1), (dict(dtype=1), 1), (dict(dtype=1, q_scale=P + 1), 1),
    (dict(seqlens_k=None), 1), (dict(block_table=None), 1), (dict(block_table=P + 2), 1), (dict(cu_seqlens_q=P + 2), 1),
    (dict(max_pages_per_seq=0), 1), (dict(total_q=(1 << 26) + 1, cu_seqlens_q=P), 2),
])
def test_attn_refusals(fp, over, code):
    assert attn(fp, q=query(fp, **over)) == code


def test_attn_refuses_caches_and_buffers(fp):
    assert attn(fp, out=None) == 1 and attn(fp, out=P + 2) == 1 and attn(fp, lse=P + 2) == 1
    assert attn(fp, scratch=None) == 3 and attn(fp, scratch=P + 8) == 3 and attn(fp, scratch_bytes=0) == 3
    assert attn(fp, ws=None) == 3 and attn(fp, ws_bytes=8) == 3
    assert attn(fp, c=cache(fp, k=None)) == 1 and attn(fp, c=cache(fp, page_size=24)) == 2
    assert attn(fp, c=cache(fp, dtype=1)) == 1 and attn(fp, c=cache(fp, d=64)) == 2
    assert attn(fp, q=query(fp, total_q=0, cu_seqlens_q=P, q=None), out=None) == 0
    L = fp.lib()
    assert L.fp_cache_attn_scratch_bytes(cache(fp), query(fp)) >= 16
    assert L.fp_cache_attn_scratch_bytes(cache(fp), query(fp, max_q=2)) == 0
    assert L.fp_cache_attn_scratch_bytes(cache(fp, page_size=24), query(fp)) == 0

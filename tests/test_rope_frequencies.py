"""The scalings' values between their ends, and what their bounds are by default."""
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def fp():
    from block_sparse_long_fp_gb300 import build, fprefill
    build.build()
    return fprefill


def mixed(f, keep, factor):
    return f * keep + f / factor * (1 - keep)


def test_ramp(fp):
    """4096 positions, base 10000, 128 dims: pairs 20.94 and 45.03 make 32 waves and 1, rounded outwards to 20
    and 46 the ends of the ramp."""
    f = [10000.0 ** (-i / 64) for i in range(64)]
    for waves, pair in ((32, 20.94), (1, 45.03)):
        assert math.isclose(4096 / (2 * math.pi) * 10000.0 ** (-pair / 64), waves, rel_tol=2e-3)
    keep = [1.0 if i <= 20 else 0.0 if i >= 46 else 1 - (i - 20) / 26 for i in range(64)]
    want = [mixed(f[i], keep[i], 8.0) for i in range(64)]
    assert np.allclose(fp.rope_frequencies(128, 10000.0, "ramp", 8.0, 4096, 1.0, 32.0), want, rtol=1e-13)
    assert np.allclose(fp.rope_frequencies(128, 10000.0, "ramp", 8.0), want, rtol=1e-13)
    assert not np.allclose(fp.rope_frequencies(128, 10000.0, "ramp", 8.0, high=4.0), want, rtol=1e-3)


def test_smooth(fp):
    f = [500000.0 ** (-i / 64) for i in range(64)]
    keep = [min(1.0, max(0.0, (8192 * x / (2 * math.pi) - 1) / 3)) for x in f]
    assert sum(0 < k < 1 for k in keep) >= 5
    want = [mixed(x, k, 8.0) for x, k in zip(f, keep)]
    assert np.allclose(fp.rope_frequencies(128, 500000.0, "smooth", 8.0, 8192, 1.0, 4.0), want, rtol=1e-13)
    assert np.allclose(fp.rope_frequencies(128, 500000.0, "smooth", 8.0, 8192), want, rtol=1e-13)


@pytest.mark.parametrize("bad", [dict(low=32.0), dict(low=40.0), dict(high=1.0), dict(low=0.0)])
def test_refusals(fp, bad):
    with pytest.raises(fp.FprefillError):
        fp.rope_frequencies(scaling="ramp", **bad)

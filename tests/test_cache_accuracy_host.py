"""The accuracies that the header states for rotary positions and the paged cache's attention, against the
arithmetic of the roundings they come from."""
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fprefill.h")


@pytest.fixture(scope="module")
def stated():
    """The header's words without line breaks and comment stars."""
    with open(HEADER) as f:
        return re.sub(r"\s*\n \*\s*", " ", f.read())


def bounds(stated, pattern):
    found = re.findall(pattern, stated)
    assert len(found) == 1, f"{pattern}: {found}"
    return [2.0 ** -int(n) for n in (found[0] if isinstance(found[0], tuple) else found)]


def halves(lo, hi, bits):
    """Midpoints between neighbours of `bits` significant bits, and numbers just beside them, over lo .. hi."""
    m = (2 ** (bits - 1) + np.arange(2 ** (bits - 1)) + 0.5) / 2 ** (bits - 1)
    x = np.concatenate([m, m * (1 - 2.0 ** -20), m * (1 + 2.0 ** -20)])
    return (x[None] * 2.0 ** np.arange(lo, hi)[:, None]).ravel().astype(np.float32)


def test_weights(stated):
    to_bf16, to_fp16, fp16_least = bounds(stated, r"to bf16 for a bf16 cache \(2\^-(\d+) of each at most\), to fp16 for an e4m3 one "
                                                  r"\(2\^-(\d+) of each, or 2\^-(\d+) of the row's largest where that is more\)")
    w = halves(-60, 15, 8)                             # the largest weight of a row lies between 2^10 and 2^14
    err = np.abs(torch.from_numpy(w).to(torch.bfloat16).double().numpy() - w.astype(np.float64))
    assert np.all(err <= to_bf16 * w) and np.any(err > to_bf16 / 2 * w)
    w = halves(-60, 15, 11)
    err = np.abs(torch.from_numpy(w).to(torch.float16).double().numpy() - w.astype(np.float64))
    for largest in (2.0 ** 10, 2.0 ** 14):
        some = w <= largest
        assert np.all(err[some] <= np.maximum(to_fp16 * w[some], fp16_least * largest))
    assert np.any(err > to_fp16 / 2 * w)


def test_queries_of_an_e4m3_cache(stated):
    """Every bf16 significand from the row's largest down to 2^-20 of it, largests from both ends of a binade."""
    exact, rest = bounds(stated, r"exact down to 2\^-(\d+) of the row's largest element, the rest to 2\^-(\d+) of it")
    x = (2.0 ** np.arange(-20, 1)[:, None] * (1 + np.arange(128) / 128)).ravel()

    def e4m3(v):
        return torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    worst = 0.0
    for largest in (1.0, 1 + 64 / 128, 1 + 127 / 128):
        y = x[x <= largest] * 128                       # the largest into 2^7 .. 2^8
        hi = e4m3(y)
        err = np.abs(hi + e4m3(y - hi) - y) / (128 * largest)
        assert np.all(err[y >= exact * 128 * largest] == 0)
        assert np.all(err <= rest)
        worst = max(worst, err.max())
    assert worst > rest / 2


def test_angles(stated):
    kept, rounded = bounds(stated, r"Angles are kept to 2\^-(\d+) of a turn at any int32 position \(negative ones too\), and rounded "
                                   r"to fp32, by 2\^-(\d+) of a turn at most")
    assert kept == 2.0 ** -32                           # the upper half of 64 bits
    rng = np.random.default_rng(0)
    t = np.concatenate([rng.integers(-2 ** 31, 2 ** 31, 100000), 2 ** 30 + np.arange(64, 4096, 64), [-2 ** 31, 2 ** 31 - 1]])
    err = np.abs(t.astype(np.int32).astype(np.float32).astype(np.float64) - t) / 2.0 ** 32
    assert np.all(err <= rounded) and np.any(err > rounded / 2)

"""Logits so large that an fp32 holds them to whole numbers at best, over the 4-bit cache: a row's weights then all
belong to its largest."""
import numpy as np
import pytest

import test_cache_gpu as tc

pytestmark = pytest.mark.gpu
fp = tc.fp


@pytest.mark.parametrize("size", [2.0 ** e for e in (24, 29, 30, 30.5, 31, 31.5, 34, 60)])
@pytest.mark.parametrize("lq,n", [(1, 700), (6, 3000)])
def test_far_logits(fp, size, lq, n):
    """Key t points along one dim with 1 .. 15 sixteenths of it, only one key that all rows attend with 16.  The next
    logit is a sixteenth of size / 11 away, so that all weight is that key's."""
    import torch
    h, g, page = 2, 4, 64
    rng = np.random.default_rng(n)
    pool = -(-n // page)
    sixteenths = rng.integers(1, 16, pool * page)
    best = int(rng.integers(0, n - lq + 1))
    sixteenths[best] = 16
    k = torch.zeros((pool * page, h, 128))
    k[:, :, 5] = torch.from_numpy(sixteenths / 16.0).float()[:, None]
    v = torch.randn((pool * page, h, 128), generator=torch.Generator().manual_seed(n))
    c = fp.QCache.empty(pool, page, h)
    slots = tc.i32(np.arange(pool * page))
    c.write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), slots)
    q = torch.zeros((lq, g * h, 128))
    q[:, :, 5] = size
    out, lse = c.attn(q.to(torch.bfloat16).cuda(), tc.i32(np.arange(pool)[None]), tc.i32([n]), max_q=lq)
    kr, vr = c.read(slots[best:best + 1])
    want = tc.host(vr).repeat(g, 1)
    # the output's rounding and the read value's (2^-8 each), and a weight's products with the group's step and least
    # value in fp16 (2^-11 each, of magnitudes up to thrice the largest)
    tol = 2.0 ** -7 * np.abs(want) + 6 * 2.0 ** -11 * np.abs(tc.host(vr)).max()
    assert np.all(np.abs(tc.host(out) - want) <= tol)
    logit = float(q[0, 0, 5].to(torch.bfloat16)) * tc.host(kr)[0, 0, 5] / np.sqrt(128)
    assert np.all(np.abs(lse.double().cpu().numpy() - logit) <= 2.0 ** -8 * logit)       # the read key is rounded

"""Logits so large that an fp32 holds them to whole numbers at best: a row's weights then all belong to its largest."""
import math

import numpy as np
import pytest

import test_cache_gpu as tc

pytestmark = pytest.mark.gpu
fp = tc.fp


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq,n", [(1, 700), (80, 700), (200, 3000), (40, 30000)])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 31, 2.0 ** 34, 2.0 ** 60, -2.0 ** 34])
def test_far_logits(fp, size, lq, n, dtype):
    """Key t points along one dim with 1 .. 15 sixteenths of it, only one key that all rows attend with 16 (the
    last for negative sizes: then the smallest counts): logits of `size` times that.  The next logit is a sixteenth
    of size / 11 away, so that all weight is that key's: 2^(least of them, in base 2) is below 2^-130."""
    import torch
    h, g, page = 2, 4, 64
    rng = np.random.default_rng(int(math.log2(abs(size))) + n)
    pool = -(-n // page)
    sixteenths = rng.integers(1, 16, n)
    if size < 0:
        sixteenths += 1                                # 2 .. 16
    best = int(rng.integers(0, n - lq + 1))
    sixteenths[best] = 16 if size > 0 else 1
    k = torch.zeros((pool * page, h, 128))
    k[:n, :, 5] = torch.from_numpy(sixteenths / 16.0).float()[:, None]
    v = torch.randn((pool * page, h, 128), generator=torch.Generator().manual_seed(n))
    q = torch.zeros((lq, g * h, 128))
    each = 2.0 ** (math.log2(abs(size)) / 2)
    q[:, :, 5] = math.copysign(each, size)
    ks = vs = None
    if dtype == "e4m3":
        ks, vs = torch.full((h,), each), torch.full((h,), 0.01)
        kc, vc = k.to(torch.float8_e4m3fn), (v / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn)
        want = vc[best].double() * np.float64(np.float32(0.01))
        ks, vs = ks.cuda(), vs.cuda()
    else:
        kc, vc = (k * each).to(torch.bfloat16), v.to(torch.bfloat16)
        want = vc[best].double()
    c = fp.KVCache(kc.view(pool, page, h, 128).cuda(), vc.view(pool, page, h, 128).cuda(), ks, vs)
    table = tc.i32(np.arange(pool)[None])
    out, lse = c.attn(q.to(torch.bfloat16).cuda(), table, tc.i32([n]), max_q=lq)
    want = want.numpy()[None, :, None, :].repeat(g, 2).reshape(1, g * h, 128)
    qe = float(q[0, 0, 5].to(torch.bfloat16))
    ke = float(kc[best, 0, 5].double()) * (each if dtype == "e4m3" else 1.0)
    # the weight is rounded by 2^-8 in the sum of values and not in its own, then the output is
    assert np.all(np.abs(tc.host(out) - want) <= (2.0 ** -7 + 2.0 ** -20) * np.abs(want))
    logit = qe * ke / math.sqrt(128)
    assert np.all(np.abs(lse.double().cpu().numpy() - logit) <= 2.0 ** -21 * abs(logit))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq", [40, 200])
def test_keys_that_share_a_far_maximum(fp, dtype, lq):
    """By tiles every one of them has the same weight: the mean of their values."""
    import torch
    h, g, n = 1, 8, 2000
    rng = np.random.default_rng(lq)
    k = torch.zeros((2048, h, 128))
    k[:, :, 3] = 0.5
    best = np.sort(rng.choice(n - lq, 5, replace=False))
    k[best, :, 3] = 1.0
    v = torch.randn((2048, h, 128), generator=torch.Generator().manual_seed(lq))
    q = torch.full((lq, g, 128), 0.0)
    q[:, :, 3] = 2.0 ** 36
    if dtype == "e4m3":
        one = torch.ones(h, device="cuda")
        c = fp.KVCache(*(x.to(torch.float8_e4m3fn).view(32, 64, h, 128).cuda() for x in (k, v)), one, one)
        vv = v.to(torch.float8_e4m3fn).float()
    else:
        c = fp.KVCache(*(x.to(torch.bfloat16).view(32, 64, h, 128).cuda() for x in (k, v)))
        vv = v.to(torch.bfloat16).float()
    out, lse = c.attn(q.to(torch.bfloat16).cuda(), tc.i32(np.arange(32)[None]), tc.i32([n]), max_q=lq)
    want = vv[best].double().mean(0).numpy()[None].repeat(lq, 0).repeat(g, 1)
    reach = vv[best].double().abs().mean(0).numpy()[None]
    assert np.all(np.abs(tc.host(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * reach)     # its rounding, and the weights'
    logit = 2.0 ** 36 / math.sqrt(128) + math.log(5)
    assert np.all(np.abs(lse.double().cpu().numpy() - logit) <= 2.0 ** -21 * logit)

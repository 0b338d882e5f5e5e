"""The status word, and kernels that stop: waits that run out or are called off."""
import numpy as np
import pytest

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


def pages(fp, tokens, h=2, page=128, seed=0):
    """A bf16 cache of one request whose pages lie in order, and its table."""
    import torch
    n = -(-tokens // page)
    torch.manual_seed(seed)
    k, v = (torch.randn((n, page, h, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    return fp.KVCache(k, v), torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)


def test_a_wait_that_runs_out_is_recorded_over_bad_device_data(fp):
    """Bad device data leaves results defined, a wait that ran out does not: the status tells of the wait."""
    cache, _ = pages(fp, 300)
    k = cache.k_cache.view(-1, 2, 128)[:3].clone()
    cache.append(k, k, i32([0, -7, 2]))
    assert cache.device_status() == fp.FP_ERR_DEVICE_BOUNDS
    fp._check(fp.lib().fp_check_wait_timeout(cache._ws_ptr, 1_000_000, fp._stream_handle()), "fp_check_wait_timeout")
    assert cache.device_status() == fp.FP_ERR_TIMEOUT
    cache.append(k, k, i32([0, -7, 2]))                # and it stays
    assert cache.device_status() == fp.FP_ERR_TIMEOUT
    cache.reset_status()
    assert cache.device_status() == 0


LONG = 262144                                          # tokens: 3 ms for a tile's way through them


def long_chunk(fp, dtype):
    """A chunk of 1024 rows, 32 heads of one KV head, whose thread blocks hold whole tiles: (cache, call)."""
    import torch
    cache, table = pages(fp, LONG, 1)
    if dtype == "e4m3":
        ones = torch.ones(1, device="cuda")
        cache = fp.KVCache(cache.k_cache.to(torch.float8_e4m3fn), cache.v_cache.to(torch.float8_e4m3fn), ones, ones)
    q = torch.randn((1024, 32, 128), device="cuda").to(torch.bfloat16)
    lens = i32([LONG])
    return cache, lambda **kw: cache.attn(q, table, lens, max_q=1024, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_waits_that_span_an_item_have_its_time(fp, dtype):
    """The limit is a tenth of the time that the walk and the loaders wait for a tile's last keys."""
    import torch
    cache, call = long_chunk(fp, dtype)
    out, lse = call()
    assert cache.device_status() == 0
    try:
        fp.lib().fp_set_wait_limit_ns(300_000)
        again, lse_again = call()
        assert cache.device_status() == 0
    finally:
        fp.lib().fp_set_wait_limit_ns(0)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


@pytest.mark.parametrize("limit", [2 ** 64 - 1, 2 ** 64 - 64000 * 2305])
def test_a_limit_without_end(fp, limit):
    """What waits that span an item are given beside the limit (64 us for each of this call's 2305 blocks of
    tokens and rows) does not turn a limit of centuries into none."""
    import torch
    cache, call = long_chunk(fp, "bf16")
    out, lse = call()
    try:
        fp.lib().fp_set_wait_limit_ns(limit)
        again, lse_again = call()
        assert cache.device_status() == 0
    finally:
        fp.lib().fp_set_wait_limit_ns(0)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_called_off_while_it_runs(fp, dtype):
    """FP_ERR_TIMEOUT recorded while tiles are on their way (as by another block, or a call on another stream):
    they stop, later calls leave their rows alone, and after a reset the same call gives the same bits."""
    import time
    import torch
    cache, call = long_chunk(fp, dtype)
    want, want_lse = call()
    outs = [torch.full_like(want, 3.0) for _ in range(20)]
    stopped = torch.tensor([fp.FP_ERR_TIMEOUT], dtype=torch.int32).pin_memory()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for out in outs:                                   # some 3 ms each
        call(out=out)
    time.sleep(0.001)
    with torch.cuda.stream(side):
        cache._ws[:1].copy_(stopped, non_blocking=True)
    torch.cuda.synchronize()
    assert cache.device_status() == fp.FP_ERR_TIMEOUT
    assert bool((outs[-1] == 3).all())
    cache.reset_status()
    out, lse = call(out=outs[0])
    assert cache.device_status() == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_a_cache_is_ready_for_any_stream(fp):
    """The status is zero when the constructor returns, whatever its stream has still to do and whatever its
    memory held: tiles look at it before they work."""
    import torch
    old, table = pages(fp, 300)
    q, lens = torch.randn((300, 8, 128), device="cuda").to(torch.bfloat16), i32([300])
    want, _ = old.attn(q, table, lens, max_q=300)
    built, used = torch.cuda.Stream(priority=-1), torch.cuda.Stream()
    with torch.cuda.stream(used):                      # memory of this stream's for the call below: none is allocated there
        out = torch.full_like(q, 3.0)
        lse = fp.KVCache(old.k_cache, old.v_cache).attn(q, table, lens, max_q=300)[1]
    torch.cuda.synchronize()
    with torch.cuda.stream(built):
        held = [torch.full((64,), fp.FP_ERR_TIMEOUT, dtype=torch.int32, device="cuda") for _ in range(64)]
        places = {t.data_ptr() for t in held}
        del held
        torch.cuda._sleep(40_000_000)                  # some 20 ms
        cache = fp.KVCache(old.k_cache, old.v_cache)
    with torch.cuda.stream(used):
        cache.attn(q, table, lens, max_q=300, out=out, lse=lse)
    torch.cuda.synchronize()
    assert cache._ws_ptr in places                     # or the test tells nothing
    assert cache.device_status() == 0
    assert torch.equal(out, want)

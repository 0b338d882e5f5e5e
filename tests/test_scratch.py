"""The attentions' scratch: one for each stream, whatever the cache."""
import threading
import time
import types

import pytest

P = 4096                                  # a non-null, aligned address that nothing reads


@pytest.fixture(scope="module")
def fp():
    from block_sparse_long_fp_gb300 import build, fprefill
    build.build()
    return fprefill


def stand_in(fp, kind, entry, stream, index=0, capturing=False):
    """A cache whose library call is `entry`, on a stream of that handle; no GPU is touched."""
    import torch
    cuda = types.SimpleNamespace(is_current_stream_capturing=lambda: capturing)
    c = object.__new__(kind)
    c.__dict__.update(_torch=types.SimpleNamespace(cuda=cuda, empty=torch.empty, uint8=torch.uint8), device="cpu", _index=index,
                      _stream=lambda _: stream, _f=(entry,), _ws_ptr=P)
    return c


@pytest.fixture
def scratch(fp, monkeypatch):
    """The table of this process, empty for the test."""
    table = {}
    monkeypatch.setattr(fp._Cache, "_scratch", table, raising=False)
    return table


def test_caches_share_a_streams_scratch(fp, scratch):
    """A cache a layer: their calls on one stream take the memory of the largest, and not of each."""
    given = []

    def entry(*args):
        given.append(args[-5:-3])
        return fp.FP_OK
    layers = [stand_in(fp, kind, entry, 7) for kind in (fp.KVCache, fp.QCache, fp.KVCache)]
    for n in (5000, 3000, 4000):
        for c in layers:
            c._attn((b"", b"", P, 0), n)
    assert len({at for at, _ in given}) == 1 and [n for _, n in given] == [5000] * 3 + [3000] * 3 + [4000] * 3
    for other in (dict(stream=8), dict(stream=7, index=1)):       # another stream, the same handle of another device
        stand_in(fp, fp.KVCache, entry, **other)._attn((b"", b"", P, 0), 5000)
        assert given[-1][0] not in {at for at, _ in given[:-1]}
    assert len(scratch) == 3
    kept = {k: s.memory for k, s in scratch.items()}
    stand_in(fp, fp.KVCache, entry, 7, capturing=True)._attn((b"", b"", P, 0), 5000)
    assert given[-1][0] not in {at for at, _ in given[:-1]} and all(scratch[k].memory is m for k, m in kept.items())
    with pytest.raises(fp.FprefillError):
        bad = stand_in(fp, fp.KVCache, lambda *a: fp.FP_ERR_WORKSPACE, 7)
        bad._attn_name = "fp_cache_attn"
        bad._attn((b"", b"", P, 0), 10)


def test_threads_of_two_caches_on_one_stream_enqueue_one_at_a_time(fp, scratch):
    busy, met = set(), []

    def entry(*args):                      # stands in for the library: enqueues, waits, enqueues
        at = args[-5]
        met.append(at in busy)
        busy.add(at)
        time.sleep(0.002)
        busy.discard(at)
        return fp.FP_OK
    caches = [stand_in(fp, kind, entry, 7) for kind in (fp.KVCache, fp.QCache)]
    threads = [threading.Thread(target=lambda c=c: [c._attn((b"", b"", P, 0), 1000) for _ in range(20)]) for c in caches * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(met) == 80 and not any(met) and len(scratch) == 1


@pytest.mark.gpu
def test_layers_on_one_stream_take_the_memory_of_one(fp):
    """Caches of eight layers, called in turn: the same results, and 40 MB of scratch once."""
    import torch
    torch.manual_seed(0)
    k, v = (torch.randn((64, 64, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((300, 16, 128), device="cuda").to(torch.bfloat16)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    lens = torch.tensor([4096], dtype=torch.int32, device="cuda")
    layers = [fp.KVCache(k, v) for _ in range(8)]
    want, _ = layers[0].attn(q, table, lens, max_q=300)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    outs = [c.attn(q, table, lens, max_q=300, want_lse=False)[0] for c in layers]
    # an output may count up to 1 MB more: the allocator does not split what would leave less; seven scratches of
    # 152 blocks, 2 x 256 rows of 128 floats each, would be 279 MB
    assert torch.cuda.memory_allocated() - before <= 8 * (want.numel() * 2 + (1 << 20))
    for out in outs:
        assert torch.equal(out, want)

"""Chunk attention and forks on the GPU in the batches that the other tests leave out: as many sequences as a cache
holds, and two caches at once on two streams."""

import pytest
import torch

from asymmetric_bit_kv_b200 import CacheConfig, KVCache
from attention_reference import assert_within, attend, cached_tokens
from test_gpu_chunk import SCALE, make, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("batch", [64, 512])
def test_many_sequences(batch, window):
    """Every launch table full: ragged lengths, some without cached and some without new tokens."""
    cache = KVCache(CacheConfig(1, batch, 4, 1, 128, 1300, 64, 64, 64, torch.bfloat16, [2], [4], page_blocks=2,
                                pool_pages=11 * batch))
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(batch)
    held = [(37 * b) % 700 if b % 5 else 0 for b in range(batch)]
    k, v, _ = tokens(sum(held), cfg, gen)
    cache.append(0, k, v, held)
    lens = [0 if b % 7 == 3 else 1 + (b * b) % 9 if b % 3 else (53 * b) % 300 for b in range(batch)]
    k, v, q = tokens(sum(lens), cfg, gen)
    out = cache.chunk_attention(0, k, v, q, lens, out_dtype=torch.float32, softmax_scale=SCALE, window=window)
    off = 0
    for b, t in enumerate(lens):
        if t:
            ck, cv = cached_tokens(cache, 0, b)
            kk, vv = torch.cat([ck, k[off:off + t].double()]), torch.cat([cv, v[off:off + t].double()])
            ref = attend(q[off:off + t], kk, vv, held[b], SCALE, window)
            assert_within(out[off:off + t], ref, SCALE, cfg, f"sequence {b} ({held[b]} cached, {t} new)")
        off += t
    assert cache.device_errors() == 0
    cache.close()


def test_two_caches_on_two_streams():
    gen = torch.Generator(device="cuda").manual_seed(5)
    caches, calls, want = [], [], []
    for fmt in ("k2v4_g64", "bq2"):
        cache = make(fmt, 3, cap=9000)
        k, v, _ = tokens(9000, cache.cfg, gen)
        cache.append(0, k, v, [6000, 3000])
        x = tokens(400, cache.cfg, gen)
        caches.append(cache)
        calls.append((*x, [300, 100]))
        want.append(cache.chunk_attention(0, *calls[-1], softmax_scale=SCALE))
    streams = [torch.cuda.Stream() for _ in caches]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for cache, call, out, stream in zip(caches, calls, outs, streams):
            cache.chunk_attention(0, *call, softmax_scale=SCALE, out=out, stream=stream)
            cache.fork_sequence(0, [2], stream=stream)
    torch.cuda.synchronize()
    for cache, out, w in zip(caches, outs, want):
        assert torch.equal(out, w) and cache.device_errors() == 0
        assert all(torch.equal(a, b) for a, b in zip(cache.dequant(0, 0, 0, 6000), cache.dequant(0, 2, 0, 6000)))
        cache.close()

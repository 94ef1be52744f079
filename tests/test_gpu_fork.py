"""Forked sequences on the GPU: copies equal to their source, independent of it afterwards, sharing pages."""

import ctypes

import pytest
import torch

from asymmetric_bit_kv_b200 import CacheConfig, KVCache, KvqError
from asymmetric_bit_kv_b200 import kvq as K
from test_gpu_chunk import FORMATS, SCALE, make, tokens

pytestmark = pytest.mark.gpu


def content(cache, layer, seq):
    n = sum(cache.lengths(layer, seq)) + cache.sinks(layer, seq)
    return (cache.lengths(layer, seq), cache.value_lengths(layer, seq), cache.sinks(layer, seq),
            *(x.cpu() for x in cache.dequant(layer, seq, 0, n)))


def same(a, b):
    return all(torch.equal(x, y) if torch.is_tensor(x) else x == y for x, y in zip(a, b))


@pytest.mark.parametrize("held", [0, 1, 5, 100, 777, 1300])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_copies_equal_their_source_and_go_their_own_way(fmt, held):
    layers = 3
    cache = make(fmt, 5, cap=2048, layers=layers)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(2)
    for layer in range(layers):
        k, v, _ = tokens(held + 250 + 40, cfg, gen)
        cache.append(layer, k, v, [held, 250, 0, 40])  # sequence 1 is overwritten, 3 is not
    before = [[content(cache, layer, b) for b in range(5)] for layer in range(layers)]
    cache.fork_sequence(0, [1, 4, 2])
    for layer in range(layers):
        for b in (0, 1, 4, 2):
            assert same(content(cache, layer, b), before[layer][0]), (layer, b)
        assert same(content(cache, layer, 3), before[layer][3])
    # a twin that appended the same tokens to every sequence by itself
    twin = make(fmt, 5, cap=2048, layers=layers)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for layer in range(layers):
        k, v, _ = tokens(held + 250 + 40, cfg, gen)
        p = (k[:held], v[:held])
        cat = lambda i: torch.cat([p[i], p[i], p[i], (k, v)[i][held + 250:], p[i]])  # noqa: E731
        twin.append(layer, cat(0), cat(1), [held, held, held, 40, held])
    for step, lens in enumerate([[1, 1, 1, 1, 1], [cfg.residual + 9, 3, 0, 70, 2 * cfg.group_k], [1, 64, 90, 0, 200]]):
        for layer in range(layers):
            k, v, _ = tokens(sum(lens), cfg, gen)
            cache.append(layer, k, v, lens)
            twin.append(layer, k, v, lens)
            q = tokens(5, cfg, gen)[2]
            for b in range(5):
                assert same(content(cache, layer, b), content(twin, layer, b)), (step, layer, b)
            assert torch.equal(cache.decode_attention(layer, q), twin.decode_attention(layer, q))
    cache.close()
    twin.close()


def _paged(pool, batch=4, layers=2, P=2):
    return KVCache(CacheConfig(layers, batch, 8, 2, 128, 2048, 64, 64, 64, torch.bfloat16, [4] * layers, [2] * layers,
                               page_blocks=P, pool_pages=pool))


def test_pages_are_shared_counted_and_returned():
    # 64 * 11 + 64 tokens: 11 blocks of 64, five full pages of 2 blocks and one half
    cache = _paged(pool=6 + 3 + 1)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(4)
    toks = []
    for layer in range(2):
        k, v, _ = tokens(64 * 12, cfg, gen)
        cache.append(layer, k, v, [64 * 12])
        toks.append((k, v))
    first = [content(cache, layer, 0) for layer in range(2)]
    for _ in range(3):  # forking again gives back what the destinations held
        cache.fork_sequence(0, [1, 2, 3])
    # 6 + 3 pages are taken: one is left, and a fork after release takes it from the pool
    cache.release_sequence(0)
    for layer in range(2):
        for b in (1, 2, 3):
            assert same(content(cache, layer, b), first[layer])
    # the source's own last page returned: two free; growing sequence 1 by two pages fits, by three does not
    k, v, _ = tokens(64 * 7, cfg, gen)
    with pytest.raises(KvqError) as e:
        cache.append(0, k, v, [0, 64 * 7])  # 18 blocks: 9 pages, 3 more than held
    assert e.value.status == K.KVQ_ERR_CAPACITY
    cache.append(0, k[:64 * 5], v[:64 * 5], [0, 64 * 5])  # 16 blocks: 8 pages
    for b in (2, 3):
        assert same(content(cache, 0, b), first[0])
    cache.release_sequence(1)
    cache.release_sequence(2)
    assert same(content(cache, 0, 3), first[0]) and same(content(cache, 1, 3), first[1])
    cache.release_sequence(3)
    # every page is back: the whole pool can be taken again
    for layer in range(2):
        k, v, _ = tokens(64 * 21, cfg, gen)
        cache.append(layer, k, v, [64 * 21])
    cache.reset()
    k, v, _ = tokens(64 * 21, cfg, gen)
    cache.append(0, k, v, [0, 64 * 21])
    cache.close()


def test_a_pool_too_small_changes_nothing():
    cache = _paged(pool=6 + 2)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(6)
    for layer in range(2):
        k, v, _ = tokens(64 * 12 + 10, cfg, gen)
        cache.append(layer, k, v, [64 * 12, 10] if layer == 0 else [64 * 2, 10])
    before = [[content(cache, layer, b) for b in range(4)] for layer in range(2)]
    with pytest.raises(KvqError) as e:
        cache.fork_sequence(0, [1, 2, 3])
    assert e.value.status == K.KVQ_ERR_CAPACITY
    for layer in range(2):
        for b in range(4):
            assert same(content(cache, layer, b), before[layer][b])
    cache.fork_sequence(0, [1, 2])
    for layer in range(2):
        for b in (1, 2):
            assert same(content(cache, layer, b), before[layer][0])
    # a copy of a copy, onto its own source's other copy
    cache.fork_sequence(1, [2])
    assert same(content(cache, 0, 2), before[0][0])
    cache.close()


def test_many_layers_and_destinations():
    # more layers and destinations than one launch takes
    layers, batch = 35, 70
    cache = KVCache(CacheConfig(layers, batch, 1, 1, 128, 256, 32, 32, 32, torch.float16, [2] * layers,
                                [2, 4, 8, 4, 2] * 7, page_blocks=2, pool_pages=200))
    gen = torch.Generator(device="cuda").manual_seed(8)
    for layer in range(layers):
        k, v, _ = tokens(150, cache.cfg, gen)
        cache.append(layer, k, v, [0, 0, 150])
    cache.fork_sequence(2, [b for b in range(batch) if b != 2])
    for layer in (0, 1, 2, 31, 32, 34):
        want = content(cache, layer, 2)
        for b in (0, 1, 63, 64, 65, 69):
            assert same(content(cache, layer, b), want), (layer, b)
    cache.close()


def test_refusals():
    cache = make("k2v4_g64", 4)
    gen = torch.Generator(device="cuda").manual_seed(10)
    k, v, _ = tokens(200, cache.cfg, gen)
    cache.append(0, k, v, [200])
    want = content(cache, 0, 0)
    for src, dsts in ((-1, [1]), (4, [1]), (0, [0]), (0, [1, 0]), (0, [1, 1]), (0, [4]), (0, [-1])):
        with pytest.raises(KvqError) as e:
            cache.fork_sequence(src, dsts)
        assert e.value.status == K.KVQ_ERR_INVALID_ARG
    lib = cache.lib
    assert lib.kvq_fork_sequence(cache.handle, 0, None, 1, 0) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_fork_sequence(cache.handle, 0, (ctypes.c_int32 * 1)(1), -1, 0) == K.KVQ_ERR_INVALID_ARG
    n = cache.kernel_launches()
    cache.fork_sequence(0, [])  # no destinations: nothing to do
    assert cache.kernel_launches() == n
    assert same(content(cache, 0, 0), want) and cache.lengths(0, 1) == (0, 0)
    cache.close()


def test_samples_of_a_prompt_decode_together():
    """The operators in a row: a prompt in chunks, forked, each sample stepping inside a window."""
    from attention_reference import assert_within, attend, cached_tokens
    from kvq_testutil import assert_attention_close

    for fmt in ("k4v2_g64_paged", "bq2", "k2v2_g32_mha"):
        cache = make(fmt, 4)
        cfg = cache.cfg
        gen = torch.Generator(device="cuda").manual_seed(12)
        for t in (200, 333, 64, 1):
            k, v, q = tokens(t, cfg, gen)
            ck, cv = cached_tokens(cache, 0, 0)
            out = cache.chunk_attention(0, k, v, q, [t], out_dtype=cfg.kv_dtype, window=250)
            ref = attend(q, torch.cat([ck, k.double()]), torch.cat([cv, v.double()]), ck.shape[0], SCALE, 250, cfg.sink_tokens)
            assert_within(out, ref, SCALE, cfg, fmt)
            cache.append(0, k, v, [t])
        cache.fork_sequence(0, [1, 2, 3])
        for _ in range(5):
            k, v, q = tokens(4, cfg, gen)
            out = cache.decode_step_window(0, k, v, q, 250, softmax_scale=SCALE)
            for b in range(4):
                ck, cv = cached_tokens(cache, 0, b)
                ref = attend(q[b:b + 1], ck, cv, ck.shape[0] - 1, SCALE, 250, cfg.sink_tokens)[0][0]
                assert_attention_close(out[b].cpu().numpy(), ref.cpu().numpy(), f"{fmt} sample {b}")
        cache.close()


@pytest.mark.parametrize("paged", [False, True])
def test_a_launch_that_fails_changes_nothing(paged):
    """On a stream whose capture was invalidated no kernel is enqueued: the call says so, and the lengths and pages
    are what they were."""
    cudart = ctypes.CDLL("libcudart.so.12")
    cache = _paged(pool=30) if paged else make("k2v4_g64", 4, cap=2048, layers=2)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(14)
    for layer in range(2):
        k, v, _ = tokens(64 * 13, cfg, gen)
        cache.append(layer, k, v, [64 * 11, 100, 64 * 2 - 100])
    cache.fork_sequence(1, [3])
    before = [[content(cache, layer, b) for b in range(4)] for layer in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert cudart.cudaStreamBeginCapture(handle, 2) == 0  # relaxed: this stream only
    try:
        assert cudart.cudaStreamSynchronize(handle) != 0  # not allowed in a capture, and the end of it
        n = cache.kernel_launches()
        with pytest.raises(KvqError) as e:
            cache.fork_sequence(0, [1, 2, 3], stream=side)
        assert e.value.status == K.KVQ_ERR_CUDA and cache.kernel_launches() == n
    finally:
        cudart.cudaStreamEndCapture(handle, ctypes.byref(graph))
        cudart.cudaGetLastError()
    for layer in range(2):
        for b in range(4):
            assert same(content(cache, layer, b), before[layer][b]), (layer, b)
    cache.fork_sequence(0, [1, 2, 3])  # and it works when it can
    for layer in range(2):
        for b in (1, 2, 3):
            assert same(content(cache, layer, b), before[layer][0])
    cache.close()


@pytest.mark.parametrize("residual,residual_v", [(192, 64), (64, 256)])
def test_pages_that_hold_only_keys_or_values_yet(residual, residual_v):
    """Separate key and value windows in pages: a shared page may hold blocks whose keys (or values) are still in the
    rings, and every sequence that shares it completes them."""
    make_one = lambda: KVCache(CacheConfig(1, 4, 8, 2, 128, 4096, 64, 64, residual, torch.bfloat16, [4], [2], residual_v=residual_v,  # noqa: E731
                                           page_blocks=2, pool_pages=120))
    cache, twin = make_one(), make_one()
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(residual)
    k, v, _ = tokens(1111, cfg, gen)
    cache.append(0, k, v, [1111])
    assert cache.lengths(0, 0)[0] != cache.value_lengths(0, 0)[0]
    cache.fork_sequence(0, [1, 2, 3])
    twin.append(0, k.repeat(4, 1, 1), v.repeat(4, 1, 1), [1111] * 4)
    for lens in ([0, 70, 300, 1], [130, 1, 0, 65], [64, 64, 64, 0]):
        k, v, q = tokens(sum(lens), cfg, gen)
        for c in (cache, twin):
            c.append(0, k, v, lens)
        q = tokens(4, cfg, gen)[2]
        for b in range(4):
            assert same(content(cache, 0, b), content(twin, 0, b)), (lens, b)
        assert torch.equal(cache.decode_attention(0, q), twin.decode_attention(0, q))
        assert torch.equal(cache.decode_attention_window(0, q, 300), twin.decode_attention_window(0, q, 300))
        if lens[0]:
            cache.release_sequence(0)
            twin.release_sequence(0)
    cache.close()
    twin.close()

"""Chunk attention on the GPU: new tokens over the packed cache and causally over themselves, against 64 bits.

Every cache format the library builds, both cache types, 1 to 8 query heads per KV head, contiguous and paged,
sliding windows, chunks from no token to several tiles, and caches from empty to many blocks. The tolerance is the
error that the kernel's roundings can cause, element by element (attention_reference.bound).
"""

import ctypes

import pytest
import torch

from asymmetric_bit_kv_b200 import CacheConfig, KVCache, KvqError
from asymmetric_bit_kv_b200 import kvq as K
from attention_reference import assert_within, attend, cached_tokens

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5

# (k bits, v bits, group_k, group_v, residual, dtype, query heads per KV head, k_axis, hadamard, sinks, page blocks)
FORMATS = {
    "k2v4_g64": (2, 4, 64, 64, 128, torch.bfloat16, 4, 0, 0, 0, 0),
    "k2v2_g32_mha": (2, 2, 32, 32, 128, torch.bfloat16, 1, 0, 0, 0, 0),
    "k2v2_g128": (2, 2, 128, 128, 128, torch.float16, 4, 0, 0, 0, 0),
    "k4v2_g64_paged": (4, 2, 64, 64, 64, torch.bfloat16, 8, 0, 0, 0, 3),
    "k8v8_g32_gv32": (8, 8, 32, 32, 64, torch.float16, 2, 0, 0, 3, 0),
    "k4v4_g32_gv128": (4, 4, 32, 128, 32, torch.float16, 2, 0, 0, 8, 1),
    "k8v2_g128_gv64": (8, 2, 128, 64, 256, torch.bfloat16, 1, 0, 0, 0, 2),
    "bq2": (2, 2, 64, 128, 128, torch.bfloat16, 4, 1, 1, 4, 0),
    "tok_k4v8_gv32": (4, 8, 128, 32, 128, torch.float16, 2, 1, 0, 0, 0),
    "rot_channel_k4v4": (4, 4, 64, 64, 64, torch.float16, 4, 0, 1, 2, 4),
    "rot_tok_k8v4_g32": (8, 4, 32, 64, 64, torch.bfloat16, 8, 1, 1, 0, 0),
    "split_windows": (2, 4, 64, 64, 192, torch.bfloat16, 4, 0, 0, 2, 0),
}


def make(fmt, batch, cap=8192, layers=1, heads=2):
    kb, vb, G, Gv, R, dt, g, ax, rot, S, P = FORMATS[fmt]
    extra = dict(page_blocks=P, pool_pages=batch * (-(-cap // (G * P)) + 1)) if P else {}
    if fmt == "split_windows":
        extra["residual_v"] = 64
    return KVCache(CacheConfig(layers, batch, heads * g, heads, 128, cap, G, Gv, R, dt, [kb] * layers, [vb] * layers,
                               sink_tokens=S, k_axis=[ax] * layers, hadamard=rot, **extra))


def tokens(n, cfg, gen, heads=None):
    """Keys (or queries, with heads) of uneven channel magnitudes, and values."""
    h = cfg.num_kv_heads
    k = torch.randn(n, h, 128, generator=gen, device="cuda") * torch.exp(0.5 * torch.randn(1, h, 128, generator=gen, device="cuda"))
    v = torch.randn(n, h, 128, generator=gen, device="cuda")
    q = torch.randn(n, cfg.num_q_heads, 128, generator=gen, device="cuda")
    return k.to(cfg.kv_dtype), v.to(cfg.kv_dtype), q.to(cfg.kv_dtype)


def check(cache, k, v, q, lens, window=0, out_dtype=None, scale=SCALE, what="", **kw):
    """One call against 64 bits for every sequence."""
    cfg = cache.cfg
    out = cache.chunk_attention(0, k, v, q, lens, out_dtype=out_dtype or cfg.kv_dtype, softmax_scale=scale, window=window, **kw)
    off = 0
    for b, t in enumerate(lens):
        if t:
            ck, cv = cached_tokens(cache, 0, b)
            n = ck.shape[0]
            kk, vv = torch.cat([ck, k[off:off + t].double()]), torch.cat([cv, v[off:off + t].double()])
            ref = attend(q[off:off + t], kk, vv, n, scale, window, cfg.sink_tokens)
            assert_within(out[off:off + t], ref, scale, cfg, f"{what} seq {b} ({n} cached, {t} new)")
        off += t
    assert cache.device_errors() == 0
    return out


@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_chunks_of_a_growing_cache(fmt):
    cache = make(fmt, 4)
    gen = torch.Generator(device="cuda").manual_seed(7)
    R = cache.cfg.residual
    # empty and tiny caches, rings not yet full, one token, no token, chunks past one tile, odd lengths
    for step, lens in enumerate([[5, 1, 0, 130], [R - 3, 2, 1, 257], [1, R + 77, 300, 1], [64, 0, 129, 33], [1, 1, 1, 1]]):
        k, v, q = tokens(sum(lens), cache.cfg, gen)
        check(cache, k, v, q, lens, what=f"step {step}")
        cache.append(0, k, v, lens)
    cache.close()


@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 127, 128, 129, 500, 1 << 29, 2 ** 31 - 1])
@pytest.mark.parametrize("fmt", ["k2v4_g64", "k4v4_g32_gv128", "bq2", "k2v2_g32_mha", "split_windows", "rot_channel_k4v4"])
def test_sliding_window(fmt, window):
    cache = make(fmt, 3)
    gen = torch.Generator(device="cuda").manual_seed(11)
    held = [700, 3, 0]
    k, v, _ = tokens(sum(held), cache.cfg, gen)
    cache.append(0, k, v, held)
    lens = [201, 40, 300]
    k, v, q = tokens(sum(lens), cache.cfg, gen)
    check(cache, k, v, q, lens, window=window)
    cache.close()


@pytest.mark.parametrize("fmt", ["k2v4_g64", "k2v2_g32_mha", "k4v2_g64_paged", "bq2", "k8v8_g32_gv32"])
def test_few_rows_over_a_long_cache(fmt):
    cache = make(fmt, 2)
    gen = torch.Generator(device="cuda").manual_seed(13)
    k, v, _ = tokens(8000, cache.cfg, gen)
    cache.append(0, k, v, [7000, 1000])
    for lens in ([1, 1], [3, 5], [0, 17], [33, 1]):
        k, v, q = tokens(sum(lens), cache.cfg, gen)
        check(cache, k, v, q, lens, what=str(lens))
    k, v, q = tokens(6, cache.cfg, gen)
    check(cache, k, v, q, [5, 1], window=3000, what="window")
    cache.close()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["k2v4_g64", "k2v2_g128", "split_windows"])
def test_output_types(fmt, out_dtype):
    cache = make(fmt, 2)
    gen = torch.Generator(device="cuda").manual_seed(17)
    k, v, _ = tokens(600, cache.cfg, gen)
    cache.append(0, k, v, [500, 100])
    k, v, q = tokens(150, cache.cfg, gen)
    check(cache, k, v, q, [100, 50], out_dtype=out_dtype)
    k, v, q = tokens(2, cache.cfg, gen)
    check(cache, k, v, q, [1, 1], out_dtype=out_dtype)
    cache.close()


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3, 1e-3])
@pytest.mark.parametrize("fmt", ["k2v4_g64", "bq2", "k2v2_g128"])
def test_softmax_scales(fmt, scale):
    cache = make(fmt, 1)
    gen = torch.Generator(device="cuda").manual_seed(19)
    k, v, _ = tokens(400, cache.cfg, gen)
    cache.append(0, k, v, [400])
    k, v, q = tokens(70, cache.cfg, gen)
    check(cache, k, v, q, [70], scale=scale)
    cache.close()


@pytest.mark.parametrize("fmt", ["k2v4_g64", "k2v2_g128"])
def test_large_and_small_queries(fmt):
    # queries of very different sizes in one call: rows are scaled on their own
    cache = make(fmt, 1)
    gen = torch.Generator(device="cuda").manual_seed(23)
    k, v, _ = tokens(500, cache.cfg, gen)
    cache.append(0, k, v, [500])
    k, v, q = tokens(64, cache.cfg, gen)
    q[:16] = (q[:16].float() * 2000).to(q.dtype)
    q[16:32] = (q[16:32].float() * 1e-4).to(q.dtype)
    q[32:40] = 0
    check(cache, k, v, q, [64], scale=1e-4)
    cache.close()


def test_scores_that_grow_along_the_sequence():
    # the running maximum rises at every tile, by much and by little
    for step in (0.02, 0.5):
        cache = make("k2v2_g128", 1)
        cfg = cache.cfg
        gen = torch.Generator(device="cuda").manual_seed(29)
        n, t = 1400, 300
        k, v, q = tokens(n + t, cfg, gen)
        u = torch.randn(128, generator=gen, device="cuda")
        u /= u.norm()
        k = (0.1 * k.float() + step / 8 * torch.arange(n + t, device="cuda")[:, None, None] * u).to(cfg.kv_dtype)
        q = (8.0 * u + 0.1 * q.float()).to(cfg.kv_dtype)
        cache.append(0, k[:n], v[:n], [n])
        check(cache, k[n:], v[n:], q[n:], [t], scale=0.125)
        cache.close()


def test_writes_exactly_its_rows_on_a_side_stream():
    cache = make("k2v4_g64", 3)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(31)
    k, v, _ = tokens(900, cfg, gen)
    cache.append(0, k, v, [300, 500, 100])
    lens = [7, 0, 140]
    k, v, q = tokens(147, cfg, gen)
    want = check(cache, k, v, q, lens)
    pad, row = 4, cfg.num_q_heads * 128
    buf = torch.full(((147 + 2 * pad) * row,), 7.5, dtype=cfg.kv_dtype, device="cuda")
    out = buf[pad * row:(pad + 147) * row].view(147, cfg.num_q_heads, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cache.chunk_attention(0, k, v, q, lens, out=out, stream=side)
    side.synchronize()
    assert got is out and torch.equal(got, want)
    assert (buf[:pad * row] == 7.5).all() and (buf[(pad + 147) * row:] == 7.5).all()
    cache.close()


def test_captured_call_replays():
    for lens in ([3, 1], [200, 90]):  # split over the cache, and not
        cache = make("k2v4_g64", 2)
        gen = torch.Generator(device="cuda").manual_seed(37)
        k, v, _ = tokens(4000, cache.cfg, gen)
        cache.append(0, k, v, [3500, 500])
        k, v, q = tokens(sum(lens), cache.cfg, gen)
        want = check(cache, k, v, q, lens)
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.chunk_attention(0, k, v, q, lens, out=out)
        k2, v2, q2 = tokens(sum(lens), cache.cfg, gen)
        for new in ((k, v, q), (k2, v2, q2)):
            for a, b in zip((k, v, q), new):
                a.copy_(b)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, cache.chunk_attention(0, k, v, q, lens, out_dtype=out.dtype))
        assert not torch.equal(out, want)
        cache.close()


@pytest.mark.parametrize("fmt", ["k2v4_g64", "k2v2_g32_mha", "k2v2_g128"])
@pytest.mark.parametrize("held", [0, 200])
def test_a_long_first_chunk_of_few_heads(fmt, held):
    """Cut into ranges by an average tile count that the first rows, which see little, do not reach: some of their
    ranges are empty."""
    cache = make(fmt, 1)
    gen = torch.Generator(device="cuda").manual_seed(43)
    k, v, _ = tokens(held, cache.cfg, gen)
    cache.append(0, k, v, [held])
    k, v, q = tokens(3500, cache.cfg, gen)
    check(cache, k, v, q, [3500])
    cache.close()


def test_repeats_and_leaves_the_cache_alone():
    cache = make("k4v2_g64_paged", 2)
    gen = torch.Generator(device="cuda").manual_seed(41)
    k, v, _ = tokens(1500, cache.cfg, gen)
    cache.append(0, k, v, [1400, 100])
    before = [x.clone() for b in range(2) for x in cache.dequant(0, b, 0, [1400, 100][b])]
    k, v, q = tokens(20, cache.cfg, gen)
    a = cache.chunk_attention(0, k, v, q, [4, 16], out_dtype=torch.float32)
    b = cache.chunk_attention(0, k, v, q, [4, 16], out_dtype=torch.float32)
    assert torch.equal(a, b)
    after = [x for b in range(2) for x in cache.dequant(0, b, 0, [1400, 100][b])]
    assert all(torch.equal(x, y) for x, y in zip(before, after))
    assert cache.lengths(0, 0)[0] + cache.lengths(0, 0)[1] == 1400
    cache.close()


def test_garbage_past_a_sequence_is_not_read():
    # the ring slots and input rows behind a sequence hold NaN
    cache = make("k2v4_g64", 1)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(43)
    lay = cache.layout(0)
    nan = torch.full((cfg.num_kv_heads * cfg.residual * 128,), float("nan"), dtype=cfg.kv_dtype, device="cuda")
    for ptr in (lay.ring_k, lay.ring_v):
        off = ptr - cache.arena.data_ptr()
        cache.arena[off:off + nan.numel() * 2].copy_(nan.view(torch.uint8))
    k, v, _ = tokens(37, cfg, gen)
    cache.append(0, k, v, [37])
    k, v, q = tokens(40, cfg, gen)
    k[21:], v[21:], q[21:] = float("nan"), float("nan"), float("nan")
    out = cache.chunk_attention(0, k[:21], v[:21], q[:21], [21], out_dtype=torch.float32)
    ck, cv = cached_tokens(cache, 0, 0)
    ref = attend(q[:21], torch.cat([ck, k[:21].double()]), torch.cat([cv, v[:21].double()]), 37, SCALE)
    assert_within(out, ref, SCALE, cfg)
    cache.close()


def test_refusals():
    cache = make("k2v4_g64", 2)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(47)
    k, v, q = tokens(5, cfg, gen)
    call = lambda *a, **kw: cache.chunk_attention(0, *a, **kw)  # noqa: E731
    for bad in ([2, 2], [2, 4], [-1, 6], [1, 2, 2]):
        with pytest.raises((ValueError, KvqError)):
            call(k, v, q, bad)
    with pytest.raises(ValueError):
        call(k.float(), v, q, [2, 3])
    with pytest.raises(ValueError):
        call(k, v, q.cpu(), [2, 3])
    with pytest.raises(ValueError):
        call(k, v, q.transpose(0, 1), [2, 3])
    with pytest.raises(ValueError):
        call(k, v, q, [2, 3], out=torch.empty(5, 4, 128, device="cuda"))
    with pytest.raises(ValueError):
        call(k, v, q, [2, 3], out_dtype=torch.float64)
    for kw in (dict(window=-1), dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf"))):
        with pytest.raises(KvqError) as e:
            call(k, v, q, [2, 3], **kw)
        assert e.value.status == K.KVQ_ERR_INVALID_ARG
    with pytest.raises(KvqError):
        cache.chunk_attention(1, k, v, q, [2, 3])
    lib, lens = cache.lib, (ctypes.c_int32 * 2)(2, 3)
    args = lambda kp, n=lens, b=2: (cache.handle, 0, kp, v.data_ptr(), q.data_ptr(), q.data_ptr(), K.KVQ_BF16, 1.0, n, b, 0, 0)  # noqa: E731
    assert lib.kvq_chunk_attention(*args(k.data_ptr() + 2)) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_chunk_attention(*args(None)) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_chunk_attention(*args(k.data_ptr(), None)) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_chunk_attention(*args(k.data_ptr(), (ctypes.c_int32 * 2)(2, 1 << 30))) == K.KVQ_ERR_INVALID_ARG
    # nothing to do is no error
    none = cache.chunk_attention(0, k[:0], v[:0], q[:0], [0, 0])
    assert none.shape == (0, cfg.num_q_heads, 128)
    assert cache.kernel_launches() == 0
    cache.close()

"""Decode of forked sequences on the GPU: pages that neighbouring sequences share are read once for all of them."""

import pytest
import torch

from asymmetric_bit_kv_b200 import CacheConfig, KVCache
from attention_reference import assert_within, attend, cached_tokens
from test_gpu_chunk import tokens

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5
BF16, FP16 = torch.bfloat16, torch.float16
# key and value bits, token group, value group, ring, dtype, KV heads, query heads per KV head, key axis, rotation,
# sinks, blocks per page
FORMATS = {
    "k2v4_g64": (2, 4, 64, 64, 128, BF16, 8, 4, 0, 0, 0, 4),
    "k2v2_g32_mha": (2, 2, 32, 32, 128, BF16, 16, 1, 0, 0, 0, 3),  # 96 positions to a page: the last tile is cut
    "k8v2_g128": (8, 2, 128, 64, 128, FP16, 8, 8, 0, 0, 2, 1),
    "bq2": (2, 2, 64, 128, 64, BF16, 8, 2, 1, 1, 4, 5),
}


def make(fmt, batch, cap):
    kb, vb, G, Gv, R, dt, heads, g, ax, rot, S, P = FORMATS[fmt]
    return KVCache(CacheConfig(1, batch, heads * g, heads, 128, cap, G, Gv, R, dt, [kb], [vb], sink_tokens=S, k_axis=[ax],
                               hadamard=rot, page_blocks=P, pool_pages=6 * (-(-cap // (G * P)) + 1) + 8 * batch))


def check_one(cache, b, q, out, what="", scale=SCALE):
    k, v = cached_tokens(cache, 0, b)
    ref = attend(q[b:b + 1], k, v, k.shape[0] - 1, scale, 0, cache.cfg.sink_tokens)
    assert_within(out[b:b + 1], ref, scale, cache.cfg, f"{what} sequence {b} of {k.shape[0]} tokens")


def check(cache, q, out, what, scale=SCALE):
    for b in range(q.shape[0]):
        check_one(cache, b, q, out, what, scale)
    assert cache.device_errors() == 0


def launches(cache, call):
    before = cache.kernel_launches()
    out = call()
    return cache.kernel_launches() - before, out


@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_runs_of_copies(fmt):
    """Two prompts' copies with others before, between and behind them, then on their own ways."""
    batch = 40
    cache = make(fmt, batch, 17000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(5)
    lens = [0] * batch
    lens[0], lens[1], lens[19], lens[20], lens[39] = 300, 16200, 0, 9333, 1
    k, v, _ = tokens(sum(lens), cfg, gen)
    cache.append(0, k, v, lens)
    cache.fork_sequence(1, range(2, 19))   # 1 .. 18
    cache.fork_sequence(20, range(21, 37))  # 20 .. 36
    cache.fork_sequence(1, [37, 38])
    q = tokens(batch, cfg, gen)[2]
    n, out = launches(cache, lambda: cache.decode_attention(0, q, out_dtype=cfg.kv_dtype, softmax_scale=SCALE))
    assert n == 3  # the shared pages, the rest, the combine
    # sequence 19 holds nothing: zeros
    assert not out[19].any()
    cache.append(0, k[:1], v[:1], [1 if b == 19 else 0 for b in range(batch)])
    out[19] = cache.decode_attention(0, q, out_dtype=cfg.kv_dtype, softmax_scale=SCALE)[19]
    check(cache, q, out, fmt)
    # steps, with flushes into pages of their own, and a few longer appends
    for t in range(3):
        more = [(7 * b + t) % 150 if b != 30 else 0 for b in range(batch)]
        k, v, _ = tokens(sum(more), cfg, gen)
        cache.append(0, k, v, more)
        k, v, q = tokens(batch, cfg, gen)
        out = cache.decode_step(0, k, v, q, out_dtype=cfg.kv_dtype, softmax_scale=SCALE)
        check(cache, q, out, f"{fmt} step {t}")
    # one of a run goes, the run falls apart around it
    cache.release_sequence(8)
    k, v, _ = tokens(700, cfg, gen)
    cache.append(0, k, v, [700 if b == 8 else 0 for b in range(batch)])
    out = cache.decode_attention(0, q, out_dtype=cfg.kv_dtype, softmax_scale=SCALE)
    check(cache, q, out, f"{fmt} after a release")
    cache.close()


def test_more_rows_than_a_tile():
    """A run of more query rows than two tiles hold, with the sequences behind the batch left alone."""
    cache = make("k8v2_g128", 80, 6400)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(6)
    k, v, _ = tokens(6000, cfg, gen)
    cache.append(0, k, v, [6000])
    cache.fork_sequence(0, range(1, 80))
    k, v, q = tokens(77, cfg, gen)
    cache.append(0, k, v, [1] * 77)
    out = torch.full((80, cfg.num_q_heads, 128), 7.0, dtype=FP16, device="cuda")
    n, _ = launches(cache, lambda: cache.decode_attention(0, q, out=out[:77], softmax_scale=SCALE))
    assert n == 3 and (out[77:] == 7.0).all()
    check(cache, q, out[:77], "77 sequences")
    cache.close()


def test_short_prompts_stay_on_the_decode_kernel():
    cache = make("k2v4_g64", 8, 2000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(7)
    k, v, _ = tokens(900, cfg, gen)
    cache.append(0, k, v, [900])
    cache.fork_sequence(0, range(1, 8))
    q = tokens(8, cfg, gen)[2]
    assert launches(cache, lambda: cache.decode_attention(0, q, softmax_scale=SCALE))[0] == 2
    cache.close()


@pytest.mark.parametrize("fmt", ["k2v4_g64", "bq2"])
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_softmax_scales(fmt, scale):
    cache = make(fmt, 24, 13000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(9)
    k, v, _ = tokens(12345, cfg, gen)
    cache.append(0, k, v, [12345])
    cache.fork_sequence(0, range(1, 24))
    k, v, q = tokens(24 * 30, cfg, gen)
    cache.append(0, k, v, [30] * 24)
    n, out = launches(cache, lambda: cache.decode_attention(0, q[:24], out_dtype=cfg.kv_dtype, softmax_scale=scale))
    assert n == 3
    check(cache, q[:24], out, f"{fmt} scale {scale}", scale)
    cache.close()


def test_copies_of_copies():
    """Copies made again over themselves and of one another: the pages' counts follow."""
    cache = make("k2v4_g64", 20, 13000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(10)
    k, v, _ = tokens(12345, cfg, gen)
    cache.append(0, k, v, [12345])
    for _ in range(3):
        cache.fork_sequence(0, range(1, 20))
        cache.fork_sequence(7, [0, 19])
        cache.fork_sequence(19, [6, 8])
        k, v, q = tokens(730, cfg, gen)
        cache.append(0, k, v, [70 if b % 2 else 3 for b in range(20)])
        out = cache.decode_attention(0, q[:20], out_dtype=cfg.kv_dtype, softmax_scale=SCALE)
        check(cache, q[:20], out, "copies of copies")
    for b in range(19):
        cache.release_sequence(b)
    out = cache.decode_attention(0, q[:20], out_dtype=cfg.kv_dtype, softmax_scale=SCALE)
    assert not out[:19].any()
    check_one(cache, 19, q, out)
    cache.close()


def test_captured_and_replayed():
    """The decode of shared pages from a graph, on another stream: the same bits as the call's."""
    cache = make("k2v4_g64", 32, 13000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(8)
    k, v, _ = tokens(12200, cfg, gen)
    cache.append(0, k, v, [12200])
    cache.fork_sequence(0, range(1, 32))
    q = tokens(32, cfg, gen)[2]
    want = cache.decode_attention(0, q, softmax_scale=SCALE)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, _ = launches(cache, lambda: cache.decode_attention(0, q, out=out, softmax_scale=SCALE))
    assert n == 3
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    cache.close()

"""Chunk attention and the decode of shared pages at full length on the GPU: no tile is left out or counted twice."""

import pytest
import torch

import lost_tiles as L
import test_gpu_fork_decode as F
from attention_reference import cached_tokens
from test_gpu_chunk import FORMATS, make, tokens

pytestmark = pytest.mark.gpu


def values(n, cfg, gen):
    """Patterned from the first token after the sinks."""
    S = cfg.sink_tokens
    v = L.patterned(n + L.TILE - S, cfg.num_kv_heads, bool(cfg.hadamard), gen)[L.TILE - S:] if S else L.patterned(n, cfg.num_kv_heads, bool(cfg.hadamard), gen)
    return v.to(cfg.kv_dtype)


@pytest.mark.parametrize("window", [0, 9000])
@pytest.mark.parametrize("held", [7000, 16200])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_chunks(fmt, held, window):
    """Single tokens (split over the cache, the slots on alternate tiles) and more than a slot's rows."""
    cache = make(fmt, 1, cap=17000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(held)
    cache.append(0, tokens(held, cfg, gen)[0], values(held, cfg, gen), [held])
    ck, cv = cached_tokens(cache, 0, 0)
    s, q = cache.sinks(0, 0), min(cache.lengths(0, 0)[0], cache.value_lengths(0, 0)[0])
    for t in (1, 70):
        k, _, x = tokens(t, cfg, gen)
        v = values(t, cfg, gen)
        out = cache.chunk_attention(0, k, v, x, [t], out_dtype=torch.float32, softmax_scale=L.SCALE, window=window)
        lo = max(0, held + t - window - s) if window else 0  # positions that every row sees
        sets = [e for e in L.tiles(s, s + q) if e.start >= s + lo]
        expanded = torch.zeros(held + t, dtype=torch.bool, device="cuda")
        expanded[s:s + q] = True
        L.assert_nothing_lost(out, x, torch.cat([ck, k.double()]), torch.cat([cv, v.double()]), held, expanded, cfg, sets,
                              f"{fmt} {t} tokens over {held}, window {window}", window)
    assert cache.device_errors() == 0
    cache.close()


@pytest.mark.parametrize("fmt,held", [("k2v4_g64", 16200), ("k8v2_g128", 12345), ("bq2", 16200), ("k2v2_g32_mha", 9270),
                                      ("k2v2_g32_mha", 9366), ("k2v2_g32_mha", 9462)])
def test_decode_of_shared_pages(fmt, held):
    """96 positions to a page of the 32-token format: the last tile ends after 32, 0 and 96 of its 128 (9270: 95 pages)."""
    copies = 24
    cache = F.make(fmt, copies, 17000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(held)
    cache.append(0, tokens(held, cfg, gen)[0], values(held, cfg, gen), [held])
    cache.fork_sequence(0, range(1, copies))
    s, page = cache.sinks(0, 0), cfg.page_blocks * cfg.group_k
    shared = cache.lengths(0, 0)[0] // page * page
    if fmt == "k2v2_g32_mha":
        assert shared % L.TILE == {9270: 32, 9366: 0, 9462: 96}[held]
    own = [1 + 3 * b for b in range(copies)]
    k, _, _ = tokens(sum(own), cfg, gen)
    cache.append(0, k, values(sum(own), cfg, gen), own)
    x = tokens(copies, cfg, gen)[2]
    n, out = F.launches(cache, lambda: cache.decode_attention(0, x, out_dtype=torch.float32, softmax_scale=L.SCALE))
    assert n == 3
    for b in range(copies):
        ck, cv = cached_tokens(cache, 0, b)
        expanded = torch.zeros(ck.shape[0], dtype=torch.bool, device="cuda")
        expanded[s:s + shared] = True
        L.assert_nothing_lost(out[b:b + 1], x[b:b + 1], ck, cv, ck.shape[0] - 1, expanded, cfg, L.tiles(s, s + shared),
                              f"{fmt} {held} copy {b}")
    assert cache.device_errors() == 0
    cache.close()

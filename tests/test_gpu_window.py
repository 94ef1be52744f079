"""Windowed decode on the GPU: the last tokens and the sinks, for every decode kernel, against 64 bits."""

import pytest
import torch

from asymmetric_bit_kv_b200 import KvqError
from asymmetric_bit_kv_b200 import kvq as K
from attention_reference import attend, cached_tokens
from kvq_testutil import assert_attention_close
from test_gpu_chunk import FORMATS, SCALE, make, tokens

pytestmark = pytest.mark.gpu


def check(cache, q, window, what=""):
    out = cache.decode_attention_window(0, q, window, out_dtype=torch.float32, softmax_scale=SCALE)
    for b in range(q.shape[0]):
        k, v = cached_tokens(cache, 0, b)
        ref = attend(q[b:b + 1], k, v, k.shape[0] - 1, SCALE, window, cache.cfg.sink_tokens)[0][0]
        assert_attention_close(out[b].cpu().numpy(), ref.cpu().numpy(), f"{what} window {window} seq {b}")
    assert cache.device_errors() == 0
    return out


@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_windows_that_end_anywhere(fmt):
    cache = make(fmt, 5)
    gen = torch.Generator(device="cuda").manual_seed(3)
    R, G = cache.cfg.residual, cache.cfg.group_k
    held = [1500, R + 3 * G + 1, 9, 1, 0]  # many blocks, a few, only the ring (and sinks), one token, none
    k, v, _ = tokens(sum(held), cache.cfg, gen)
    cache.append(0, k, v, held)
    n = cache.lengths(0, 0)[1]
    q = tokens(5, cache.cfg, gen)[2]
    # inside the ring, at its end, at block, tile and page borders, past every length
    for w in sorted({1, 2, 7, 8, 9, n - 1, n, n + 1, n + 31, n + 32, n + 63, n + 64, n + 65, n + G, n + 3 * G + 1, 1400, 1500, 5000, 2 ** 31 - 1}):
        if w >= 1:
            check(cache, q, w)
    full = cache.decode_attention(0, q, out_dtype=torch.float32, softmax_scale=SCALE)
    assert torch.equal(full, cache.decode_attention_window(0, q, 1 << 30, softmax_scale=SCALE))
    cache.close()


@pytest.mark.parametrize("fmt", ["k2v4_g64", "k2v2_g32_mha", "bq2", "k8v8_g32_gv32", "k4v2_g64_paged", "split_windows"])
def test_steps_equal_append_and_windowed_decode(fmt):
    """decode_step_window over more steps than a ring holds, against append then decode_attention_window."""
    a, b = make(fmt, 3), make(fmt, 3)
    cfg = a.cfg
    gen = torch.Generator(device="cuda").manual_seed(5)
    held = [cfg.residual + 5, 2, 0]
    k, v, _ = tokens(sum(held), cfg, gen)
    for c in (a, b):
        c.append(0, k, v, held)
    window = cfg.residual // 2 + 37
    for step in range(cfg.residual + 2 * cfg.group_k + 3):
        k, v, q = tokens(3, cfg, gen)
        w = window if step % 2 else 3 * cfg.residual // 2
        got = a.decode_step_window(0, k, v, q, w, softmax_scale=SCALE)
        b.append(0, k, v, [1, 1, 1])
        want = b.decode_attention_window(0, q, w, softmax_scale=SCALE)
        assert torch.equal(got, want) or torch.allclose(got, want, rtol=0, atol=2e-5), step
        assert a.lengths(0, 0) == b.lengths(0, 0) and a.lengths(0, 2) == b.lengths(0, 2)
        if step % 41 == 0:
            check(b, q, w, f"step {step}")
    for s in range(3):
        n = sum(a.lengths(0, s)) + a.sinks(0, s)
        for x, y in zip(a.dequant(0, s, 0, n), b.dequant(0, s, 0, n)):
            assert torch.equal(x, y)
    a.close()
    b.close()


@pytest.mark.parametrize("fmt", ["k2v4_g64", "k2v2_g32_mha", "k8v8_g32_gv32", "k2v2_g128", "tok_k4v8_gv32", "bq2"])
def test_hidden_tokens_may_hold_anything(fmt):
    """Infinite and NaN values of tokens before the window, some in the block and the ring chunk that the window
    cuts, must not reach the output."""
    for first in (302, 330, 371, 383, 400, 542, 545, 599):
        cache = make(fmt, 2)
        cfg = cache.cfg
        gen = torch.Generator(device="cuda").manual_seed(9)
        k, v, _ = tokens(1200, cfg, gen)
        for back, x in ((1, "nan"), (2, "inf"), (3, "-inf"), (10, "nan"), (37, "inf"), (100, "nan")):
            v[first - back] = float(x)  # sequence 0; sequence 1 stays finite
        cache.append(0, k, v, [600, 600])
        check(cache, tokens(2, cfg, gen)[2], 600 - first, f"first visible {first}")
        cache.close()


def test_batch_smaller_than_the_cache_and_a_side_stream():
    cache = make("k2v4_g64", 4)
    gen = torch.Generator(device="cuda").manual_seed(21)
    k, v, _ = tokens(2000, cache.cfg, gen)
    cache.append(0, k, v, [900, 600, 400, 100])
    q = tokens(2, cache.cfg, gen)[2]
    want = check(cache, q, 333)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(2, cache.cfg.num_q_heads, 128, device="cuda")
    cache.decode_attention_window(0, q, 333, out=out, softmax_scale=SCALE, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    cache.close()


def test_captured_windowed_decode_replays():
    cache = make("k2v4_g64", 2)
    gen = torch.Generator(device="cuda").manual_seed(27)
    k, v, _ = tokens(2000, cache.cfg, gen)
    cache.append(0, k, v, [1500, 500])
    q = tokens(2, cache.cfg, gen)[2]
    out = torch.empty(2, cache.cfg.num_q_heads, 128, device="cuda")
    check(cache, q, 700)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_attention_window(0, q, 700, out=out, softmax_scale=SCALE)
    q.copy_(tokens(2, cache.cfg, gen)[2])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, check(cache, q, 700))
    cache.close()


def test_refusals():
    cache = make("k2v4_g64", 2)
    k, v, q = tokens(2, cache.cfg, torch.Generator(device="cuda").manual_seed(1))
    for w in (0, -5):
        with pytest.raises(KvqError) as e:
            cache.decode_attention_window(0, q, w)
        assert e.value.status == K.KVQ_ERR_INVALID_ARG
        with pytest.raises(KvqError) as e:
            cache.decode_step_window(0, k, v, q, w)
        assert e.value.status == K.KVQ_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        cache.decode_attention_window(0, q[:, :4], 5)
    with pytest.raises(ValueError):
        cache.decode_step_window(0, k[:1], v, q, 5)
    with pytest.raises(ValueError):
        cache.decode_attention_window(0, q, 5, out=torch.empty(1, 8, 128, device="cuda"))
    with pytest.raises(KvqError):
        cache.decode_attention_window(3, q, 5)
    assert cache.lengths(0, 0) == (0, 0)  # a refused step appends nothing
    cache.close()


def test_windows_wider_than_32_bits_are_refused():
    """(not cut to their low 32 bits)"""
    cache = make("k2v4_g64", 2)
    k, v, q = tokens(2, cache.cfg, torch.Generator(device="cuda").manual_seed(1))
    cache.append(0, k, v, [1, 1])
    for w in (2 ** 32 + 5, 2 ** 31, -2 ** 32 + 7):
        with pytest.raises(ValueError, match="32 bits"):
            cache.decode_attention_window(0, q, w)
        with pytest.raises(ValueError, match="32 bits"):
            cache.decode_step_window(0, k, v, q, w)
        with pytest.raises(ValueError, match="32 bits"):
            cache.chunk_attention(0, k, v, q, [1, 1], window=w)
    assert cache.lengths(0, 0) == (0, 1)
    cache.close()

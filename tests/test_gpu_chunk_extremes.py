"""Chunk attention and the decode of shared pages on the GPU: keys and values at the ends of their type."""

import pytest
import torch

import test_gpu_fork_decode as F
from attention_reference import attend, cached_tokens
from oracle import kvq_oracle as O
from test_gpu_chunk import FORMATS, make, tokens

pytestmark = pytest.mark.gpu

SCALE = 1e-6  # keys of 6e4 and queries of 1: scores of a few units


def largest(shape, signed, cfg, gen):
    """Values from 0 (signed: from the least finite one) to 65504 (in bf16, which has no such number, 65536), both in
    every 32 tokens of every channel and in every 32 channels of every token: the largest code of many groups stands
    for more than the largest fp16 number once the group's scale has been rounded up. In a rotated cache every token
    is a row of H, so that one rotated channel is 65529 and the others 0."""
    f16 = cfg.kv_dtype == torch.float16
    top, low = 65504.0 if f16 else 65536.0, (-65504.0 if f16 else -65280.0) if signed else 0.0
    if cfg.hadamard:
        h = torch.from_numpy(O.sylvester(128)).to("cuda").double() * 5792 * 128 ** 0.5
        return h[torch.randint(128, shape[:2], generator=gen, device="cuda")].to(cfg.kv_dtype)
    x = low + (top - low) * torch.rand(shape, generator=gen, device="cuda")
    i = torch.arange(shape[0], device="cuda")[:, None, None] + torch.arange(shape[2], device="cuda")
    x = torch.where((i % 32 == 0).expand(shape), top, torch.where((i % 32 == 7).expand(shape), low, x))
    return x.to(cfg.kv_dtype)


def allowed(ref, cfg, dtype):
    """attention_reference.bound with 2^-9 in the place of 2^-11 for a rounded key or value. A value q d + m of a group
    from m >= -65504 to at most 65536 is at most 65536 + 131040 * 2^-11 < 65600, since d is off by at most half a step:
    the limit to 65504 moves it by at most 96, less than 2^-9 of it. A rotated query adds its 2^-11 to a score."""
    out, mean, size, norms, most = ref
    if cfg.hadamard:
        size, mean = most, torch.maximum(mean, norms)
    weights = torch.expm1(2.0 * SCALE * (2.0 ** -9 + 2.0 ** -11) * size)
    p = 2.0 ** -8 if cfg.kv_dtype == torch.bfloat16 else 2.0 ** -11
    err = mean * (weights + p + 2.0 ** -9 + 1e-5) + 1e-5
    return err + (out.abs() + err) * torch.finfo(dtype).eps / 2


def assert_allowed(got, ref, cfg, what):
    err, tol = (got.double() - ref[0]).abs(), allowed(ref, cfg, got.dtype)
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: {(err / tol).max().item():.3g} of what the roundings allow"


@pytest.mark.parametrize("signed", [False, True])
@pytest.mark.parametrize("fmt", sorted(set(FORMATS) - {"split_windows"}))
def test_chunks_over_the_largest_values(fmt, signed):
    cache = make(fmt, 2)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(3)
    shape = (1000, cfg.num_kv_heads, 128)
    cache.append(0, largest(shape, signed, cfg, gen), largest(shape, signed, cfg, gen), [700, 300])
    k, v, q = tokens(140, cfg, gen)
    out = cache.chunk_attention(0, k, v, q, [5, 135], out_dtype=torch.float32, softmax_scale=SCALE)
    for b, (a, e) in enumerate(((0, 5), (5, 140))):
        ck, cv = cached_tokens(cache, 0, b)
        n = ck.shape[0]
        ref = attend(q[a:e], torch.cat([ck, k[a:e].double()]), torch.cat([cv, v[a:e].double()]), n, SCALE)
        assert_allowed(out[a:e], ref, cfg, f"{fmt} sequence {b}")
    cache.close()


@pytest.mark.parametrize("copies", [1, 24])
@pytest.mark.parametrize("fmt", ["k2v4_g64", "k8v2_g128", "bq2"])
def test_decode_of_the_largest_values_alone_and_of_copies(fmt, copies):
    cache = F.make(fmt, 24, 13000)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(4)
    shape = (12345, cfg.num_kv_heads, 128)
    cache.append(0, largest(shape, False, cfg, gen), largest(shape, False, cfg, gen), [12345])
    if copies > 1:
        cache.fork_sequence(0, range(1, copies))
    q = tokens(copies, cfg, gen)[2]
    n, out = F.launches(cache, lambda: cache.decode_attention(0, q, out_dtype=torch.float32, softmax_scale=SCALE))
    assert n == (3 if copies > 1 else 2)
    k, v = cached_tokens(cache, 0, 0)
    for b in range(copies):
        assert_allowed(out[b:b + 1], attend(q[b:b + 1], k, v, k.shape[0] - 1, SCALE), cfg, f"{fmt} sequence {b} of {copies}")
    cache.close()

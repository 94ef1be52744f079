"""Chunk attention and the decode of shared pages on the GPU: keys and values at the ends of their type."""

import pytest
import torch

import test_gpu_fork_decode as F
from attention_reference import attend, bound, cached_tokens
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


BAD = (float("nan"), float("inf"), float("-inf"))


def check_rows(cache, k, v, q, lens, bad, window, what):
    """bad[b]: tokens of sequence b (cached or new) whose values, and of new ones some keys, are infinite or NaN. A row
    that sees none of them is as if they were not there; one that does is not finite."""
    cfg = cache.cfg
    out = cache.chunk_attention(0, k, v, q, lens, out_dtype=torch.float32, window=window)
    off = hidden = 0
    for b, t in enumerate(lens):
        ck, cv = cached_tokens(cache, 0, b)
        n = ck.shape[0]
        kk, vv = torch.cat([ck, k[off:off + t].double()]), torch.cat([cv, v[off:off + t].double()])
        kk[bad[b]], vv[bad[b]] = 0.0, 0.0
        assert torch.isfinite(kk).all() and torch.isfinite(vv).all()
        i, j = torch.arange(n, n + t, device="cuda")[:, None], torch.tensor(bad[b], device="cuda")[None, :]
        sees = j <= i
        if window:
            sees &= (j > i - window) | (j < cfg.sink_tokens)
        sees = sees.any(1)
        ref = attend(q[off:off + t], kk, vv, n, 128 ** -0.5, window, cfg.sink_tokens)
        got, clean = out[off:off + t], ~sees
        err, tol = (got.double() - ref[0]).abs(), bound(ref, 128 ** -0.5, cfg, torch.float32)
        assert torch.isfinite(got[clean]).all(), f"{what} sequence {b}: what a row does not see reached it"
        assert (err[clean] <= tol[clean]).all(), f"{what} sequence {b}"
        assert not torch.isfinite(got[sees]).all(-1).any(), f"{what} sequence {b}: a row hides what it sees"
        off += t
        hidden += int(clean.sum())
    assert cache.device_errors() == 0
    return hidden


def plant(x, at, gen):
    for e, i in enumerate(at):
        c = torch.randint(128, (1 + 40 * (e % 2),), generator=gen, device="cuda")
        x[i, :, c] = BAD[e % 3]


@pytest.mark.parametrize("window", [1, 16, 100, 129, 300])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_tokens_outside_the_window_may_hold_anything(fmt, window):
    hidden = 0
    for seed, lens in enumerate([[201, 300], [5, 1], [20, 33], [64, 700]]):
        cache = make(fmt, 2)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        held = [900, 5]
        k, v, _ = tokens(sum(held), cache.cfg, gen)
        S = cache.cfg.sink_tokens
        old = [900 - x for x in (1, 2, 40, 70, 127, 130, 190, 260, 299)]
        plant(v, old, gen)
        cache.append(0, k, v, held)
        k, v, q = tokens(sum(lens), cache.cfg, gen)
        new = [x for x in (0, 3, 90, 150, 199) if x < lens[0]], [x for x in (4, 64, 127, 129, 290, 650) if x < lens[1]]
        for x in (k, v):
            plant(x, [*new[0], *(lens[0] + y for y in new[1])], gen)
        bad = [old + [900 + y for y in new[0]], [5 + y for y in new[1]]]
        assert min(bad[0]) >= S and (not bad[1] or min(bad[1]) >= S)
        hidden += check_rows(cache, k, v, q, lens, bad, window, f"{fmt} window {window} {lens}")
        cache.close()
    assert hidden > 0


@pytest.mark.parametrize("held", [0, 3, 500])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_later_tokens_may_hold_anything(fmt, held):
    for seed, (lens, new) in enumerate([([400, 130], ([257, 300, 399], [129])), ([7, 30], ([6], [11, 12])), ([1, 1000], ([], [513, 999]))]):
        cache = make(fmt, 2)
        gen = torch.Generator(device="cuda").manual_seed(20 + seed)
        k, v, _ = tokens(2 * held, cache.cfg, gen)
        cache.append(0, k, v, [held, held])
        k, v, q = tokens(sum(lens), cache.cfg, gen)
        for x in (k, v):
            plant(x, [*new[0], *(lens[0] + y for y in new[1])], gen)
        check_rows(cache, k, v, q, lens, [[held + y for y in n] for n in new], 0, f"{fmt} {held} {lens}")
        cache.close()


def test_a_sink_that_is_not_finite_reaches_every_row():
    cache = make("bq2", 1)
    gen = torch.Generator(device="cuda").manual_seed(30)
    k, v, _ = tokens(800, cache.cfg, gen)
    plant(v, [2], gen)
    cache.append(0, k, v, [800])
    k, v, q = tokens(90, cache.cfg, gen)
    assert check_rows(cache, k, v, q, [90], [[2]], 130, "sink") == 0
    cache.close()

"""Decode on the GPU over rings whose slots past the newest token hold what older tokens left there: it must not matter.

A ring is read in chunks of 8 slots. The slots behind the newest token in its chunk keep the keys and values of tokens a
ring's length back, which a window hides, or of a sequence that was released.
"""

import pytest
import torch

from test_gpu_chunk import FORMATS, SCALE, make, tokens
from test_gpu_window import check

pytestmark = pytest.mark.gpu


def spoil(x, at):
    for e, i in enumerate(at):
        x[i] = (float("nan"), float("inf"), float("-inf"))[e % 3]


@pytest.mark.parametrize("held", [601, 604, 607])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_hidden_tokens_that_a_ring_still_holds(fmt, held):
    """Values only: a key that is not finite spoils its channel's group of tokens, seen ones among them."""
    cache = make(fmt, 2)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(held)
    k, v, _ = tokens(held, cfg, gen)
    s = cfg.sink_tokens
    # the positions whose slots follow the newest token's
    R = {cfg.residual, cfg.residual_v or cfg.residual}
    spoil(v, [p for r in R for p in range(held - r, held - r + 8) if p >= s])
    for i in range(0, held, 30):  # (what passes a ring in one append is never written to it)
        cache.append(0, k[i:i + 30], v[i:i + 30], [min(30, held - i), 0])
    q = tokens(2, cfg, gen)[2]
    for window in (1, 5, min(R) - 9):
        check(cache, q, window, f"{fmt} {held}")
    k, v, q = tokens(2, cfg, gen)
    got = cache.decode_step_window(0, k, v, q, 5, softmax_scale=SCALE)
    assert torch.isfinite(got).all()
    cache.close()


@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_what_a_released_sequence_left(fmt):
    cache = make(fmt, 2)
    cfg = cache.cfg
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v, _ = tokens(40, cfg, gen)
    spoil(k, range(0, 40, 2))
    spoil(v, range(40))
    cache.append(0, k, v, [20, 20])
    cache.release_sequence(0)
    k, v, _ = tokens(13, cfg, gen)
    cache.append(0, k, v, [13, 0])
    cache.release_sequence(1)
    for n in (1, 3, 6):
        k, v, _ = tokens(n, cfg, gen)
        cache.append(0, k, v, [0, n])
        q = tokens(2, cfg, gen)[2]
        check(cache, q, 2 ** 30, f"{fmt} {n}")
        check(cache, q, 2, f"{fmt} {n}")
        want = cache.decode_attention_window(0, q, 2 ** 30, softmax_scale=SCALE)
        assert torch.equal(cache.decode_attention(0, q, softmax_scale=SCALE), want)
    cache.close()

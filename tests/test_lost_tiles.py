"""The inputs of lost_tiles.py do show a tile that is left out: planted in the reference, without a GPU."""

import types

import pytest
import torch

import lost_tiles as L


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("n", [3000, 7040, 16200])
def test_a_tile_left_out_of_the_reference_is_seen(n, rotated):
    cfg = types.SimpleNamespace(hadamard=int(rotated), sink_tokens=0, kv_dtype=torch.bfloat16)
    gen = torch.Generator().manual_seed(n)
    k = torch.randn(n, 1, 128, generator=gen).double()
    v = L.patterned(n, 1, rotated, gen, "cpu")
    q = torch.randn(3, 4, 128, generator=gen)
    expanded = torch.arange(n) < n - 200
    whole = L.mean(q, k, v, n - 3)[1]
    got = whole.reshape(1, 3, 4, 128).transpose(0, 1).reshape(3, 4, 128).float()
    L.assert_nothing_lost(got, q, k, v, n - 3, expanded, cfg, L.tiles(0, n - 200), "whole")
    for lost in (slice(0, 128), slice(1280, 1408), slice(n - 328, n - 200), slice(n - 264, n - 200)):
        rest = torch.ones(n, dtype=torch.bool)
        rest[lost] = False
        p, _ = L.mean(q, k, v, n - 3)
        p = p * rest
        out = torch.einsum("hrn,nhd->hrd", p / p.sum(-1, keepdim=True), v)
        got = out.reshape(1, 3, 4, 128).transpose(0, 1).reshape(3, 4, 128).float()
        with pytest.raises(AssertionError, match="of what the roundings allow"):
            L.assert_nothing_lost(got, q, k, v, n - 3, expanded, cfg, [], "a tile less")

"""Chunk attention, windowed decode and forks without a GPU: what is refused on the host, before any CUDA call."""

import ctypes

import pytest
import torch

from asymmetric_bit_kv_b200 import load_library
from asymmetric_bit_kv_b200 import kvq as K


def test_a_null_cache_is_refused_on_the_host():
    lib = load_library()
    lens = (ctypes.c_int32 * 1)(1)
    assert lib.kvq_chunk_attention(None, 0, None, None, None, None, 0, 1.0, lens, 1, 0, None) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_decode_attention_window(None, 0, None, None, 0, 1.0, 1, 8, None) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_decode_step_window(None, 0, None, None, None, None, 0, 1.0, 1, 8, None) == K.KVQ_ERR_INVALID_ARG
    assert lib.kvq_fork_sequence(None, 0, lens, 1, None) == K.KVQ_ERR_INVALID_ARG
    assert b"null" in lib.kvq_last_error()


def test_the_binding_checks_shapes_and_types():
    t = torch.zeros(2, 3)
    with pytest.raises(ValueError, match="shape"):
        K._need_shape(t, (2, 4), "k")
    with pytest.raises(ValueError, match="CUDA"):
        K._need(t, torch.float32, "k")
    with pytest.raises(ValueError, match="not supported"):
        K.KVCache._out_like(t, None, torch.float64)
    with pytest.raises(ValueError, match="not supported"):
        K.KVCache._out_like(t, torch.zeros(2, 3, dtype=torch.int32), torch.float32)

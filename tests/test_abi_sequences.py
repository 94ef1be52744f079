"""Chunk attention, windowed decode and forks without a GPU: what is refused on the host, before any CUDA call."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

from asymmetric_bit_kv_b200 import CacheConfig, load_library, required_bytes
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


def test_the_workspace_of_chunk_attention_is_there_where_it_is_used():
    """(the arena of a short cache, or of one with separate key and value windows, does not hold it)"""
    def size(**kw):
        base = dict(num_layers=1, max_batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_tokens=512, group_k=64,
                    group_v=64, residual=128, kv_dtype=torch.bfloat16, k_bits=[2], v_bits=[4])
        return required_bytes(CacheConfig(**{**base, **kw}))

    rows = 128 * 4 + 8  # bytes of a partial row
    assert size() < 1 << 21
    long = size(max_tokens=4096)
    assert long >= 32768 * rows  # a wave of items with one part a row
    # separate windows: what decode's parts need, 16 rows x 66 x 6, in its place
    assert size(max_tokens=4096, residual_v=64) <= long - (32768 - 16 * 66 * 6) * rows


def test_integers_wider_than_32_bits_are_refused():
    """(not cut to their low 32 bits: a copy would go to another sequence)"""
    for bad in (2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="32 bits"):
            K.lens_array([3, bad])
    assert list(K.lens_array([3, 2 ** 31 - 1, -2 ** 31])) == [3, 2 ** 31 - 1, -2 ** 31]

    class Calls:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    cache = K.KVCache.__new__(K.KVCache)
    cache.lib, cache.handle = Calls(), None
    with pytest.raises(ValueError, match="src .* 32 bits"):
        cache.fork_sequence(2 ** 32, [1])
    with pytest.raises(ValueError, match="32 bits"):
        cache.fork_sequence(0, [1, 2 ** 32 + 2])
    for call in (cache.chunk_attention, cache.decode_attention_window, cache.decode_step_window):
        args = {cache.chunk_attention: (None, None, None, [1]), cache.decode_attention_window: (None, 5),
                cache.decode_step_window: (None, None, None, 5)}[call]
        with pytest.raises(ValueError, match="layer .* 32 bits"):
            call(2 ** 32, *args)


def test_a_cache_whose_page_lists_do_not_fit_host_memory_is_refused():
    """(by a status: a C++ exception must not leave a C entry point)"""
    code = """
import ctypes, resource, sys
import torch
from asymmetric_bit_kv_b200 import CacheConfig, load_library
lib = load_library()
n = 512
c, keep = CacheConfig(n, 1, 1, 1, 128, 4096, 64, 64, 64, torch.float16, [2] * n, [2] * n, page_blocks=1, pool_pages=1 << 22).to_c()
h = ctypes.c_void_p()
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (256 << 20),) * 2)
s = lib.kvq_cache_create(ctypes.byref(c), 0x100000, 1 << 62, ctypes.byref(h))
print(s, lib.kvq_last_error().decode(), h.value)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split()[:1] == [str(K.KVQ_ERR_INVALID_ARG)] and "host memory" in r.stdout and r.stdout.strip().endswith("None")

"""Attention in 64 bits over what a cache holds, for the tests of chunk attention, windows and forks,
and the error that the kernels' roundings can cause.

The keys and values come from the cache's own fp32 reconstruction (``dequant``, checked bit for bit against
the oracle elsewhere); a Hadamard cache's quantized tokens are rotated back in 64 bits.
"""

import torch

from oracle import kvq_oracle as O


def cached_tokens(cache, layer, seq):
    """(K, V) [tokens, Hkv, D] in 64 bits on the device, and the quantized range [s, s + q) of the keys."""
    s = cache.sinks(layer, seq)
    q, n = cache.lengths(layer, seq)
    qv = cache.value_lengths(layer, seq)[0]
    k, v = (x.double() for x in cache.dequant(layer, seq, 0, s + q + n))
    if cache.cfg.hadamard:
        h = torch.from_numpy(O.sylvester(128)).double().to(k.device)
        k[s:s + q] = k[s:s + q] @ h
        v[s:s + qv] = v[s:s + qv] @ h
    return k, v


def attend(q, k, v, first, scale, window=0, sinks=0):
    """Queries q [T, Hq, D] of the tokens first, first + 1, ... over tokens k, v [n, Hkv, D]: query t sees token j
    when j <= first + t and, with a window, when also j > first + t - window or j < sinks. A token that is not seen
    takes no part, whatever it holds. Returns (out [T, Hq, D], sum_j p_j |v_j| [T, Hq, D], max_j sum_d |q_d k_jd| over
    seen tokens [T, Hq, 1], and the same two with 2-norms of whole vectors, sum_j p_j |v_j|_2 and max_j |q|_2 |k_j|_2
    [T, Hq, 1]), in 64 bits."""
    q = q.double()
    T, Hq, D = q.shape
    n, Hkv, _ = k.shape
    g = Hq // Hkv
    i = torch.arange(first, first + T, device=q.device)[:, None]
    j = torch.arange(n, device=q.device)[None, :]
    seen = j <= i
    if window:
        seen &= (j > i - window) | (j < sinks)
    some = seen.any(0)  # tokens that no query sees are dropped, so that their infinities reach nothing
    k, v, seen = k[some], v[some], seen[:, some]
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        o = torch.zeros(T, Hq, 1, device=q.device, dtype=torch.float64)
        return z, z.clone(), o, o.clone(), o.clone()
    qh = q.reshape(T, Hkv, g, D)
    z = torch.einsum("thgd,nhd->thgn", qh, k) * scale
    z = z.masked_fill(~seen[:, None, None, :], float("-inf"))
    p = torch.softmax(z, -1)
    size = torch.einsum("thgd,nhd->thgn", qh.abs(), k.abs()).masked_fill(~seen[:, None, None, :], 0.0)
    out = torch.einsum("thgn,nhd->thgd", p, v)
    mean = torch.einsum("thgn,nhd->thgd", p, v.abs())
    norms = torch.einsum("thgn,nh->thg", p, v.norm(dim=-1)).reshape(T, Hq, 1)
    most = (qh.norm(dim=-1) * k.norm(dim=-1).amax(0)[None, :, None]).reshape(T, Hq, 1)
    return out.reshape(T, Hq, D), mean.reshape(T, Hq, D), size.amax(-1, keepdim=True).reshape(T, Hq, 1), norms, most


def bound(ref, scale, cfg, out_dtype):
    """Largest error of the tensor-core kernels' outputs, element by element.

    * A dequantized key is rounded to fp16 (relative 2^-11), and so is a rotated query: each score is off by at
      most e = |scale| (2 * 2^-11) sum|q k|, and a softmax weight by a factor of at most exp(2e).
    * Each probability is rounded to fp16 (2^-11) or, next to exact bf16 values, to bf16 (2^-8), each dequantized
      value to fp16 (2^-11): a weighted mean of |v| times those. Values below fp16's normal range are off by at most
      2^-25 absolutely, a key of that kind moves a score by |scale| 2^-25 sum|q|, which 1e-5 covers here.
    * fp32 sums: 1e-5 relative to the mean of |v| covers the 128-term dot products (128 * 2^-24) and the sums over
      tokens, which add in blocks.
    * The output is rounded once: half a step of its type.
    * A Hadamard cache rounds in the rotated basis: a score is off by at most e with sum|(Hq)_d (Hk)_d| <= |q|_2 |k|_2
      in the place of sum|q k| (Cauchy-Schwarz, H orthogonal), and a value element, errors u |(Hv)_d| rotated back with
      entries 1/sqrt(D), by at most u / sqrt(D) sum_d |(Hv)_d| <= u |v|_2. The norms of a row's visible tokens bound both.
    """
    out, mean, size, norms, most = ref
    if cfg.hadamard:
        size = most
    e = abs(scale) * 2.0 ** -10 * size
    weights = torch.expm1(2.0 * e)
    p = 2.0 ** -8 if cfg.kv_dtype == torch.bfloat16 else 2.0 ** -11
    rounded = norms if cfg.hadamard else mean
    err = mean * (weights + p) + rounded * (2.0 ** -11 + 1e-5) + 1e-5
    return err + (out.abs() + err) * torch.finfo(out_dtype).eps / 2


def assert_within(got, ref, scale, cfg, what=""):
    out = ref[0]
    assert got.shape == out.shape, (got.shape, out.shape)
    err = (got.double() - out).abs()
    tol = bound(ref, scale, cfg, got.dtype)
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error is {worst:.3g} of what the roundings allow (max abs {err.max().item():.3g})"

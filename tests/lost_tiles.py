"""Attention at full length with inputs that show a tile left out or counted twice, for the tests of chunk attention
and of the decode of shared pages.

The worst case of every rounding (attention_reference.bound) is as large as the output at many thousand tokens, because
it lets every score be off by its most in the worst direction. Here scores are nearly equal (a small softmax scale), so
that the output is nearly the mean of the values, and every 128-token tile has values of one pattern, 1 and -1 per
channel, that is its own: without one of N tiles the output moves by about 1/N, and the roundings allow 2^-10.
"""

import torch

TILE = 128
SCALE = 1e-4


def patterned(n, heads, rotated, gen, device="cuda"):
    """Values [n, heads, 128]: 1 and -1, the same in every 128 tokens, drawn anew for each. Rotated caches: rows of H
    times sqrt(128), so that one rotated channel holds all of a token."""
    rows = -(-n // TILE) + 1
    if rotated:
        from oracle import kvq_oracle as O

        h = torch.from_numpy(O.sylvester(128)).to(device).double() * 128 ** 0.5
        x = h[torch.randint(128, (rows, heads), generator=gen, device=device)]
        x = x * (2.0 * torch.randint(2, (rows, heads, 1), generator=gen, device=device) - 1)
    else:
        x = 2.0 * torch.randint(2, (rows, heads, 128), generator=gen, device=device).double() - 1
    return x.repeat_interleave(TILE, 0)[:n]


def mean(q, k, v, first, window=0, sinks=0):
    """Weights p [heads of KV, T * group, n] and the output [.., 128] in 64 bits of queries q [T, Hq, 128] of the tokens
    first, first + 1, ... over k, v [n, Hkv, 128]."""
    T, Hq, D = q.shape
    n, Hkv, _ = k.shape
    i, j = torch.arange(first, first + T, device=q.device)[:, None], torch.arange(n, device=q.device)[None, :]
    seen = j <= i
    if window:
        seen &= (j > i - window) | (j < sinks)
    z = torch.einsum("thgd,nhd->htgn", q.double().reshape(T, Hkv, Hq // Hkv, D), k) * SCALE
    p = torch.softmax(z.masked_fill(~seen[None, :, None], float("-inf")), -1).reshape(Hkv, -1, n)
    return p, torch.einsum("hrn,nhd->hrd", p, v)


def rows_of(x, Hkv):
    """[T, Hq, 128] as mean()'s rows."""
    T, Hq, D = x.shape
    return x.double().reshape(T, Hkv, Hq // Hkv, D).transpose(0, 1).reshape(Hkv, -1, D)


def tolerance(p, q, k, v, out, expanded, cfg, dtype):
    """What the roundings allow, element by element. `expanded` [n]: tokens that the tensor-core kernel dequantizes to
    fp16 (half a step, 2^-11) and multiplies by an fp16 probability (2^-11). The others: exact ones with a probability
    of their type (2^-8 in bf16), or those of a forked sequence's own pages, where codes and zero points are
    multiplied apart, by rounded products p d and p m (|q d| + |m| <= 3 |x| here, 2 * 2^-11 each: 3 * 2^-10 < 2^-8). In
    a rotated cache an element of a rounded value is off by at most sum_d |(Hv)_d| / sqrt(128) in the place of |v|, and
    in the others' part by its 2-norm (Cauchy-Schwarz). A score is off by |scale| 2^-10 |q| |k| (the key's and a
    rotated query's 2^-11 each), a weight by twice that. 1e-5: fp32 sums. The output is rounded once."""
    a = v.abs()
    if cfg.hadamard:
        from oracle import kvq_oracle as O

        h = torch.from_numpy(O.sylvester(128)).to(v.device).double()
        a = torch.where(expanded[:, None, None], (v @ h).abs().sum(-1, keepdim=True) / 128 ** 0.5, v.norm(dim=-1, keepdim=True)).expand_as(v)
    size = torch.einsum("hrn,nhd->hrd", p, a)
    other = torch.einsum("hrn,nhd->hrd", p[..., ~expanded], a[~expanded])
    e = SCALE * 2.0 ** -10 * rows_of(q, k.shape[1]).norm(dim=-1, keepdim=True) * k.norm(dim=-1).amax(0)[:, None, None]
    err = 2.0 ** -10 * size + 2.0 ** -8 * other + torch.expm1(2 * e) * size + 1e-5
    return err + (out.abs() + err) * torch.finfo(dtype).eps / 2


def least_shift(p, v, out, tol, sets):
    """For tokens left out, and counted twice, the largest of what the output moves by against the tolerance: the least
    of it over `sets` of tokens (slices)."""
    worst = float("inf")
    for t in sets:
        w = p[..., t].sum(-1, keepdim=True)
        part = torch.einsum("hrn,nhd->hrd", p[..., t], v[t])
        for moved in ((out - part) / (1 - w), (out + part) / (1 + w)):
            worst = min(worst, ((moved - out).abs() / tol).max().item())
    return worst


def tiles(lo, hi):
    """The 128-token tiles from lo, the last one cut at hi."""
    return [slice(t, min(t + TILE, hi)) for t in range(lo, hi, TILE)]


def assert_nothing_lost(got, q, k, v, first, expanded, cfg, sets, what, window=0):
    p, out = mean(q, k, v, first, window, cfg.sink_tokens)
    tol = tolerance(p, q, k, v, out, expanded, cfg, got.dtype)
    shift = least_shift(p, v, out, tol, sets)
    assert shift > 2.0, f"{what}: a tile left out moves the output by {shift:.3g} of the tolerance only"
    err = (rows_of(got, k.shape[1]) - out).abs()
    assert torch.isfinite(err).all() and (err <= tol).all(), f"{what}: {(err / tol).max().item():.3g} of what the roundings allow"

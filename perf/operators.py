"""Cases of the operators that read and share a packed KV cache, and their plain forms.

Three operators of ``asymmetric_bit_kv_b200.KVCache``:

``chunk``  ``chunk_attention``: a chunk of new tokens of every sequence attends to the sequence's cached
           tokens (exact sinks, quantized blocks, exact recent tokens) and causally to the chunk itself,
           optionally inside a sliding window that leaves the sink tokens visible.
``window`` ``decode_attention_window``: one query per sequence over the last ``window`` tokens and the sinks.
``fork``   ``fork_sequence``: a cached prompt becomes several sequences (parallel samples of one prompt),
           followed by their first decode in every layer, which reads all that the copies hold.

``own`` false runs the plain form (elementary torch operations in 32 bits over unpacked codes), ``own`` true
the calls a user makes. ``exact`` computes the same outputs in 64 bits, one sequence and head at a time.
"""

import math
import random

import torch

own = False

D = 128  # channels of a head

# Cache formats, as in the repository's workloads and tests: code bits, tokens per key group, channels per
# value group, exact recent tokens, query / KV heads, and for BQ2_0 the per-token keys, rotation and sinks.
FORMATS = {
    # the GQA layer of the headline workload
    "k2v4_g64": dict(kb=2, vb=4, g=64, gv=64, res=128, hq=32, hkv=8, axis=0, rot=0, sinks=0),
    # the MHA layer with 32-token groups
    "k2v2_g32_mha": dict(kb=2, vb=2, g=32, gv=32, res=128, hq=32, hkv=32, axis=0, rot=0, sinks=0),
    # the long-context layer with 128-token groups
    "k2v2_g128": dict(kb=2, vb=2, g=128, gv=128, res=128, hq=32, hkv=8, axis=0, rot=0, sinks=0),
    # the 36-layer workload's layers: 4-bit keys, 2-bit values, and the first layers' 8-bit keys
    "k4v2_g64": dict(kb=4, vb=2, g=64, gv=64, res=64, hq=32, hkv=8, axis=0, rot=0, sinks=0),
    "k8v4_g64": dict(kb=8, vb=4, g=64, gv=64, res=64, hq=32, hkv=8, axis=0, rot=0, sinks=0),
    # BQ2_0: 2-bit keys and values per token, rotated, 4 exact first tokens
    "bq2_s4": dict(kb=2, vb=2, g=64, gv=128, res=128, hq=32, hkv=8, axis=1, rot=1, sinks=4),
    # per-channel 4-bit keys and values with 4 sinks
    "k4v4_g64_s4": dict(kb=4, vb=4, g=64, gv=64, res=128, hq=32, hkv=8, axis=0, rot=0, sinks=4),
}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # ---- a chunk of new tokens over the cache
        # one long prompt arriving in chunks: the ninth 4096-token chunk (the largest case)
        dict(name="chunk_long", op="chunk", fmt="k2v4_g64", dtype="bf16", batch=1, ctx=32768, new=4096, window=0, ragged=False, paged=0),
        # first chunk of four prompts, nothing cached yet, multi-head
        dict(name="chunk_first", op="chunk", fmt="k2v2_g32_mha", dtype="bf16", batch=4, ctx=0, new=2048, window=0, ragged=False, paged=0),
        # a serving step: ragged prompts' chunks and single tokens over ragged paged contexts
        dict(name="chunk_ragged", op="chunk", fmt="k4v2_g64", dtype="bf16", batch=8, ctx=12001, new=1021, window=0, ragged=True, paged=16),
        # a few drafted tokens of every sequence of a batch
        dict(name="chunk_draft", op="chunk", fmt="k2v4_g64", dtype="bf16", batch=16, ctx=8192, new=5, window=0, ragged=False, paged=0),
        # a sliding-window layer with sinks in fp16
        dict(name="chunk_window", op="chunk", fmt="k4v4_g64_s4", dtype="f16", batch=1, ctx=40000, new=2048, window=4096, ragged=False, paged=0),
        # short follow-up turns over the rotated per-token format
        dict(name="chunk_turn", op="chunk", fmt="bq2_s4", dtype="bf16", batch=2, ctx=8190, new=300, window=0, ragged=True, paged=0),
        # ---- one token over a window and the sinks
        # one stream, small window: launch latency
        dict(name="window_one", op="window", fmt="k4v4_g64_s4", dtype="f16", batch=1, ctx=8191, window=1024, ragged=False, paged=0),
        # a decode batch of sliding-window layers
        dict(name="window_batch", op="window", fmt="k2v4_g64", dtype="bf16", batch=32, ctx=16384, window=4096, ragged=False, paged=0),
        # ragged long contexts in pages, an odd wide window
        dict(name="window_long", op="window", fmt="k4v2_g64", dtype="bf16", batch=16, ctx=60001, window=16385, ragged=True, paged=16),
        # ---- samples of one prompt
        # three more samples of a short prompt
        dict(name="fork_few", op="fork", fmt="k2v4_g64", dtype="bf16", batch=4, ctx=1000, layers=2, paged=4),
        # fifteen more samples of a long prompt in pages
        dict(name="fork_many", op="fork", fmt="k4v2_g64", dtype="bf16", batch=16, ctx=8200, layers=8, paged=16),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cost(c):
    """(score values of the plain form, operations) of a case, to keep drawn cases inside the listed range."""
    f = FORMATS[c["fmt"]]
    t = c.get("new", 1)
    rows = c["batch"] * c.get("layers", 1) * f["hq"] * t
    return rows * (c["ctx"] + t), c["batch"] * c.get("layers", 1) * f["hkv"] * (c["ctx"] + t)


def draw(rng):
    most = [max(_cost(c)[k] for c in listed()) for k in (0, 1)]
    while True:
        op = rng.choice(("chunk", "chunk", "window", "fork"))
        c = dict(op=op, fmt=rng.choice(sorted(FORMATS)), dtype=rng.choice(("bf16", "bf16", "f16")))
        c["paged"] = rng.choice((0, 3, 16))
        if op == "chunk":
            c |= dict(batch=_log(rng, 1, 24), ctx=rng.choice((0, 1)) * rng.randrange(1, 300) if rng.random() < 0.2 else _log(rng, 300, 32768),
                      new=_log(rng, 1, 4096), window=rng.choice((0, 0, _log(rng, 16, 16384))), ragged=rng.random() < 0.5)
        elif op == "window":
            c |= dict(batch=_log(rng, 1, 48), ctx=_log(rng, 200, 60000), window=_log(rng, 16, 16384), ragged=rng.random() < 0.5)
        else:
            c |= dict(batch=rng.randrange(2, 17), ctx=_log(rng, 100, 8200), layers=rng.randrange(1, 9), paged=rng.choice((0, 4, 16)))
        if all(x <= m for x, m in zip(_cost(c), most)):
            return c


# ---------------------------------------------------------------- sizes
def _lens(c):
    """(cached tokens, new tokens) of each sequence."""
    b, ctx, new = c["batch"], c["ctx"], c.get("new", 1)
    if not c.get("ragged"):
        return [ctx] * b, [new] * b
    r = random.Random(1000003 * b + 101 * ctx + new)
    return ([ctx] + [r.randrange(0, ctx + 1) for _ in range(b - 1)],
            [new] + [r.choice((1, max(1, new // 7), r.randrange(1, new + 1))) for _ in range(b - 1)])


def _split(f, n):
    """(sinks, quantized, ring) tokens of a sequence whose n tokens were appended at once: a token that finds
    the ring of `res` tokens full moves the oldest g tokens to a quantized block."""
    s = min(f["sinks"], n)
    t = n - s
    q = 0 if t <= f["res"] else -(-(t - f["res"]) // f["g"]) * f["g"]
    return s, q, t - q


def work(case):
    f = FORMATS[case["fmt"]]
    hq, hkv, w = f["hq"], f["hkv"], case.get("window", 0)
    ctx, new = _lens(case)
    # packed bytes of one quantized token of one head: codes, and fp16 (scale, zero point) pairs
    key = D * f["kb"] / 8 + (4 * D / f["g"] if f["axis"] == 0 else 4 * D / f["gv"])
    packed = key + D * f["vb"] / 8 + 4 * D / f["gv"]
    by = fl = 0.0
    if case["op"] == "fork":
        s, q, n = _split(f, case["ctx"])
        copies = case["batch"]
        by = q * hkv * packed + copies * (s + n) * hkv * D * 4 + copies * hq * D * 4
        fl = 4.0 * copies * hq * D * case["ctx"]
        return {"bytes": by * case["layers"], "flops": fl * case["layers"]}
    for c, t in zip(ctx, new):
        if case["op"] == "window":
            t, c1 = 1, c
            first = max(0, c - w)
        else:
            c1 = c + t
            first = max(0, c + 1 - w) if w else 0
        s, q, n = _split(f, c)
        quant = max(0, s + q - max(first, s))                     # visible quantized tokens
        exact = (min(c1, s) if first > 0 else s) + min(n, c - first)  # visible exact cached tokens
        by += quant * hkv * packed + exact * hkv * D * 4 + 2 * t * hq * D * 2
        if case["op"] == "window":
            fl += 4.0 * hq * D * min(c, w + s)
        else:
            by += t * hkv * D * 4
            if w:
                fl += 4.0 * hq * D * sum(min(c + i + 1, w + f["sinks"]) for i in range(t))
            else:
                fl += 4.0 * hq * D * (t * c + t * (t + 1) / 2)
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------- inputs
def _rotate(x):
    """x . H over the last axis, H the normalized Sylvester Hadamard matrix, in fp32 butterflies."""
    x = x.float()
    shape = x.shape
    w = 1
    while w < D:
        y = x.reshape(*shape[:-1], D // (2 * w), 2, w)
        x = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), dim=-2).reshape(shape)
        w *= 2
    return x * torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32, device=x.device)


def _tokens(case, seed):
    """Raw tensors of a case: keys with per-channel magnitudes, values and queries, [tokens, heads, D]."""
    f, dt = FORMATS[case["fmt"]], DTYPES[case["dtype"]]
    ctx, new = _lens(case)
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    layers = case.get("layers", 1)
    mag = torch.exp(0.5 * normal(layers, 1, f["hkv"], D))
    held = case["ctx"] if case["op"] == "fork" else sum(ctx)
    k = (normal(layers, held, f["hkv"], D) * mag).to(dt)
    v = normal(layers, held, f["hkv"], D).to(dt)
    rows = {"chunk": sum(new), "window": case["batch"], "fork": case["batch"]}[case["op"]]
    q = normal(layers, rows, f["hq"], D).to(dt)
    kn = vn = None
    if case["op"] == "chunk":
        kn = (normal(sum(new), f["hkv"], D) * mag[0]).to(dt)
        vn = normal(sum(new), f["hkv"], D).to(dt)
    return k, v, q, kn, vn


def _codes(x, bits, dims):
    """Quantizer of the cache over the dimension `dims`: codes, fp16 scale, fp16 zero point."""
    top = float(2 ** bits - 1)
    lo, hi = x.amin(dims, keepdim=True), x.amax(dims, keepdim=True)
    d = ((hi - lo) / top).clamp_min(1e-6).half()
    m = (lo + 0.0).half()
    return ((x - m.float()) / d.float()).round().clamp(0, top).to(torch.uint8), d, m


def _pack(f, k, v, n):
    """What the cache holds of one sequence's n tokens ([n, hkv, D] each): exact sinks and recent tokens, codes
    of the others with their scales, [hkv, ...]."""
    s, q, _ = _split(f, n)
    k, v = k.transpose(0, 1), v.transpose(0, 1)
    kq, vq = k[:, s:s + q].float(), v[:, s:s + q].float()
    if f["rot"]:
        kq, vq = _rotate(kq), _rotate(vq)
    hkv = f["hkv"]
    per_token = lambda x, bits: _codes(x.reshape(hkv, q, D // f["gv"], f["gv"]), bits, 3)  # noqa: E731
    vc = per_token(vq, f["vb"]) if q else None
    kc = (per_token(kq, f["kb"]) if f["axis"] else _codes(kq.reshape(hkv, q // f["g"], f["g"], D), f["kb"], 2)) if q else None
    return dict(sk=k[:, :s], sv=v[:, :s], rk=k[:, s + q:], rv=v[:, s + q:], kc=kc, vc=vc, s=s, q=q, n=n)


def _padded(parts, most, dev):
    """[sequences, heads, most, D] from one [heads, length, D] a sequence, zeros behind each."""
    out = torch.zeros(len(parts), parts[0].shape[0], most, D, dtype=parts[0].dtype, device=dev)
    for i, p in enumerate(parts):
        out[i, :, :p.shape[1]] = p
    return out


def prepare(case, seed):
    f = FORMATS[case["fmt"]]
    ctx, new = _lens(case)
    k, v, q, kn, vn = _tokens(case, seed)
    st = dict(case=case, q=q, kn=kn, vn=vn, new=new, window=case.get("window", 0))
    layers = case.get("layers", 1)
    if own:
        import asymmetric_bit_kv_b200 as kvq

        room = max(ctx) + f["g"] + 8
        pages = {}
        if case["paged"]:
            per = lambda n: -(-(_split(f, n)[1] // f["g"]) // case["paged"])  # noqa: E731
            need = per(case["ctx"]) + 2 * case["batch"] if case["op"] == "fork" else sum(map(per, ctx))
            pages = dict(page_blocks=case["paged"], pool_pages=need + 2)
        cache = kvq.KVCache(kvq.CacheConfig(layers, case["batch"], f["hq"], f["hkv"], D, room, f["g"], f["gv"], f["res"],
                                            DTYPES[case["dtype"]], [f["kb"]] * layers, [f["vb"]] * layers, sink_tokens=f["sinks"],
                                            k_axis=[f["axis"]] * layers, hadamard=f["rot"], **pages))
        for i in range(layers):
            cache.append(i, k[i], v[i], [case["ctx"]] if case["op"] == "fork" else ctx)
        st["cache"] = cache
        st["lens"] = kvq.lens_array(new)
        return st
    dev = q.device
    if case["op"] == "fork":
        seqs = [_pack(f, k[i], v[i], case["ctx"]) for i in range(layers)]
    else:
        at = [sum(ctx[:i]) for i in range(len(ctx))]
        seqs = [_pack(f, k[0, a:a + n], v[0, a:a + n], n) for a, n in zip(at, ctx)]
    qm = max(p["q"] for p in seqs)
    blank = torch.zeros(f["hkv"], 0, D, device=dev)
    ng = D // f["gv"]

    def codes(name, axis):
        """Codes [sequences, heads, qm, D] and their scales and zero points, in groups."""
        c = _padded([(p[name][0].reshape(f["hkv"], p["q"], D) if p["q"] else blank.to(torch.uint8)) for p in seqs], qm, dev)
        shape = (f["hkv"], qm // f["g"], D) if axis == 0 else (f["hkv"], qm, ng)
        par = [torch.zeros(len(seqs), *shape, dtype=torch.float16, device=dev) for _ in range(2)]
        for i, p in enumerate(seqs):
            for j in range(2 if p["q"] else 0):
                x = p[name][1 + j].squeeze(2 if axis == 0 else 3)
                par[j][i, :, :x.shape[1]] = x
        return c, par[0], par[1]

    st["k_codes"], st["v_codes"] = codes("kc", f["axis"]), codes("vc", 1)
    rows = max(p["rk"].shape[1] for p in seqs)
    st["exact"] = [_padded([p[n] for p in seqs], m, dev) for n, m in (("sk", f["sinks"]), ("sv", f["sinks"]), ("rk", rows), ("rv", rows))]
    ints = lambda x: torch.tensor(x, device=dev)  # noqa: E731
    st["s"], st["qn"], st["n"] = ints([p["s"] for p in seqs]), ints([p["q"] for p in seqs]), ints([p["n"] for p in seqs])
    # where each new token sits in the padded batch
    if case["op"] == "chunk":
        st["seq_of"] = ints([b for b, t in enumerate(new) for _ in range(t)])
        st["tok_of"] = ints([i for t in new for i in range(t)])
    st["sinks"] = f["sinks"]
    st["H"] = _rotate(torch.eye(D, device=dev)) if f["rot"] else None
    st["seqs"] = seqs
    return st


# ---------------------------------------------------------------- plain form
def _dequant(codes, d, m, axis, g, gv):
    """q * d + m in fp32, [sequences, heads, tokens, D]."""
    b, h, n, _ = codes.shape
    x = codes.float()
    if axis == 0:
        return (x.reshape(b, h, n // g, g, D) * d.float()[:, :, :, None] + m.float()[:, :, :, None]).reshape(b, h, n, D)
    return (x.reshape(b, h, n, D // gv, gv) * d.float()[..., None] + m.float()[..., None]).reshape(b, h, n, D)


def _plain(f, window, sinks, tokens, s, qn, n, H, q, kn, vn, new):
    """softmax(q k^T / sqrt(D)) v in fp32 over padded sequences. tokens: (k codes, v codes, exact tokens);
    q [b, t, hq, D] the queries of the positions n .. n + t - 1 (new tokens kn, vn [b, t, hkv, D]) or, without new
    tokens, of the last position."""
    (kc, kd, km), (vc, vd, vm), (sk, sv, rk, rv) = tokens
    b, t, hq, _ = q.shape
    kh = _dequant(kc, kd, km, f["axis"], f["g"], f["gv"])
    vh = _dequant(vc, vd, vm, 1, f["g"], f["gv"])
    if H is not None:
        kh, vh = kh @ H, vh @ H
    dev = q.device
    ar = lambda x: torch.arange(x, device=dev)[None, :]  # noqa: E731
    s1, q1, n1 = s[:, None], qn[:, None], n[:, None]
    # position of every key in its sequence, and whether there is such a key
    pos = [ar(sk.shape[2]).expand(b, -1), s1 + ar(kh.shape[2]), s1 + q1 + ar(rk.shape[2])]
    there = [ar(sk.shape[2]) < s1, ar(kh.shape[2]) < q1, s1 + q1 + ar(rk.shape[2]) < n1]
    ks, vs = [sk.float(), kh, rk.float()], [sv.float(), vh, rv.float()]
    if kn is not None:
        pos.append(n1 + ar(t))
        there.append(ar(t) < new[:, None])
        ks.append(kn.float().transpose(1, 2))
        vs.append(vn.float().transpose(1, 2))
        at = n1 + ar(t)
    else:
        at = n1 - 1
    pos, there, ks, vs = torch.cat(pos, 1), torch.cat(there, 1), torch.cat(ks, 2), torch.cat(vs, 2)
    seen = there[:, None, :] & (pos[:, None, :] <= at[:, :, None])
    if window:
        seen &= (pos[:, None, :] > at[:, :, None] - window) | (pos[:, None, :] < sinks)
    hkv = ks.shape[1]
    # query heads of a KV head share its keys: rows [b, hkv, group * t, D]
    rows = q.float().reshape(b, t, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, D)
    w = (rows * (D ** -0.5)) @ ks.transpose(2, 3)
    w.view(b, hkv, hq // hkv, t, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w @ vs) / torch.where(total > 0, total, torch.ones_like(total))  # a row that sees nothing gives zeros
    return o.reshape(b, hkv, hq // hkv, t, D).permute(0, 3, 1, 2, 4).reshape(b, t, hq, D)


def run(st):
    case = st["case"]
    f, dt = FORMATS[case["fmt"]], DTYPES[case["dtype"]]
    if own:
        cache = st["cache"]
        if case["op"] == "chunk":
            return cache.chunk_attention(0, st["kn"], st["vn"], st["q"][0], st["lens"], window=st["window"], out_dtype=dt)
        if case["op"] == "window":
            return cache.decode_attention_window(0, st["q"][0], st["window"], out_dtype=dt)
        cache.fork_sequence(0, range(1, case["batch"]))
        return [cache.decode_attention(i, st["q"][i], out_dtype=dt) for i in range(case["layers"])]
    tokens, s, qn, n, q = (st["k_codes"], st["v_codes"], st["exact"]), st["s"], st["qn"], st["n"], st["q"]
    if case["op"] == "chunk":
        b, t = case["batch"], max(st["new"])
        where = (st["seq_of"], st["tok_of"])
        pad = lambda x: torch.zeros(b, t, *x.shape[1:], dtype=x.dtype, device=x.device).index_put_(where, x)  # noqa: E731
        new = torch.bincount(st["seq_of"], minlength=b)
        o = _plain(f, st["window"], st["sinks"], tokens, s, qn, n, st["H"], pad(q[0]), pad(st["kn"]), pad(st["vn"]), new)
        return o[where].to(dt)
    if case["op"] == "window":
        return _plain(f, st["window"], st["sinks"], tokens, s, qn, n, st["H"], q[0][:, None], None, None, None)[:, 0].to(dt)
    # every layer's prompt, copied for each sample
    c = case["batch"]
    copy = lambda x: x.repeat_interleave(c, 0)  # noqa: E731
    tokens = tuple(tuple(copy(x) for x in part) for part in tokens)
    o = _plain(f, 0, st["sinks"], tokens, copy(s), copy(qn), copy(n), st["H"], q.reshape(-1, 1, f["hq"], D), None, None, None)
    return list(o.reshape(case["layers"], c, f["hq"], D).to(dt).unbind(0))


# ---------------------------------------------------------------- 64 bits
def _values64(f, p, name):
    """Dequantized and exact tokens of one packed sequence in order, [heads, tokens, D] in 64 bits."""
    parts = [p["s" + name].double()]
    if p["q"]:
        c, d, m = p[name + "c"]
        x = (c.double() * d.double() + m.double()).reshape(f["hkv"], p["q"], D)
        if f["rot"]:
            i = torch.arange(D, device=x.device)
            bits = i[:, None] & i[None, :]
            odd = sum((bits >> e) & 1 for e in range(7)) % 2  # Sylvester: (-1)^popcount(i & j) / sqrt(D)
            x = x @ ((1.0 - 2.0 * odd.double()) / math.sqrt(D))
        parts.append(x)
    return torch.cat([*parts, p["r" + name].double()], 1)


def _attend64(q, k, v, first, window, sinks):
    """Rows q [t, group, D] at positions first, first + 1, ... over keys k, v [n, D] of one head."""
    t, n = q.shape[0], k.shape[0]
    i = torch.arange(first, first + t, device=q.device)[:, None]
    j = torch.arange(n, device=q.device)[None, :]
    hidden = j > i
    if window:
        hidden |= (j <= i - window) & (j >= sinks)
    out = torch.zeros_like(q)
    for a in range(0, t, 1024):  # rows at a time, to bound the scores held
        z = torch.einsum("tgd,nd->gtn", q[a:a + 1024], k) / math.sqrt(D)
        z.masked_fill_(hidden[None, a:a + 1024], -math.inf)
        if n:
            out[a:a + 1024] = torch.einsum("gtn,nd->tgd", torch.softmax(z, -1).nan_to_num_(0.0), v)
    return out


def exact(case, seed):
    f = FORMATS[case["fmt"]]
    ctx, new = _lens(case)
    k, v, q, kn, vn = _tokens(case, seed)
    g, w = f["hq"] // f["hkv"], case.get("window", 0)
    outs = []
    if case["op"] == "fork":
        for layer in range(case["layers"]):
            p = _pack(f, k[layer], v[layer], case["ctx"])
            kk, vv = _values64(f, p, "k"), _values64(f, p, "v")
            x = q[layer].double().reshape(case["batch"], f["hkv"], g, D)
            rows = []
            for h in range(f["hkv"]):
                z = torch.softmax(torch.einsum("bgd,nd->bgn", x[:, h], kk[h]) / math.sqrt(D), -1)
                rows.append(z @ vv[h])
            outs.append(torch.stack(rows, 1).reshape(case["batch"], f["hq"], D))
        return outs
    at = row = 0
    for n, t in zip(ctx, new):
        p = _pack(f, k[0, at:at + n], v[0, at:at + n], n)
        at += n
        kk, vv = _values64(f, p, "k"), _values64(f, p, "v")
        if case["op"] == "chunk":
            kk = torch.cat([kk, kn[row:row + t].double().transpose(0, 1)], 1)
            vv = torch.cat([vv, vn[row:row + t].double().transpose(0, 1)], 1)
            first = n
        else:
            t, first = 1, n - 1
        x = q[0, row:row + t].double().reshape(t, f["hkv"], g, D)
        row += t
        o = torch.stack([_attend64(x[:, h], kk[h], vv[h], first, w, f["sinks"]) for h in range(f["hkv"])], 1)
        outs.append(o.reshape(t, f["hq"], D))
    return torch.cat(outs, 0)

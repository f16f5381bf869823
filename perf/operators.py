"""Cases of the paged KV-cache operators: per-head norms with the position rotation
(``qk_norm_rope``), appending keys and values to the cache (``kv_append``) and attention of new
tokens over it (``paged_attention``), in a plain form of elementary torch operations and as the
library's calls.

A case is a dict of plain values: ``op`` and the sizes it needs.  A batch of ``seqs`` sequences
has ``new`` new tokens in each of its first ``chunks`` sequences and one in every other one; the
cache holds ``kv`` tokens of each sequence (new ones included), or with ``ragged`` between 1/seqs
of ``kv`` and ``kv``.  Head counts follow the 5120-wide attention projection of the benchmark's
model (40 heads of 128) with 8 key-value heads, beside generic ones.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn


def listed():
    def rope(name, tokens, q_heads, kv_heads, dim, rot, dtype, norm=True, interleaved=False):
        return {"name": name, "op": "norm_rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rot, "dtype": dtype, "norm": norm, "interleaved": interleaved}

    def append(name, seqs, new, chunks, kv, ragged, q_heads, kv_heads, dim, rot, cache, page, dtype="bf16", interleaved=False):
        return {"name": name, "op": "append", "seqs": seqs, "new": new, "chunks": chunks, "kv": kv, "ragged": ragged,
                "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "cache": cache, "page": page,
                "dtype": dtype, "interleaved": interleaved}

    def attend(name, seqs, new, chunks, kv, ragged, q_heads, kv_heads, dim, cache, page, window=0, causal=True, lse=False):
        return {"name": name, "op": "attention", "seqs": seqs, "new": new, "chunks": chunks, "kv": kv, "ragged": ragged,
                "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page, "window": window,
                "causal": causal, "lse": lse}

    return [
        # one token of one request: launch latency
        rope("rope_token", 1, 40, 8, 128, 128, "bf16"),
        # the prefill chunk of the benchmark
        rope("rope_prefill", 4096, 40, 8, 128, 128, "bf16"),
        # wide heads rotated in their first quarter only, fp32 projections, an odd token count
        rope("rope_partial_fp32", 2049, 24, 4, 256, 64, "f32", interleaved=True),
        # a decode step of 64 requests, queries in the same launch
        append("append_decode", 64, 1, 0, 8192, True, 40, 8, 128, 128, "fp8", 16),
        # a long prompt in one chunk
        append("append_prefill", 1, 8192, 1, 8192, False, 40, 8, 128, 128, "fp8", 64),
        # prompt chunks beside single tokens, bf16 cache, wide heads with partial rotation, no queries
        append("append_mixed_bf16", 33, 509, 5, 4099, True, 0, 4, 256, 64, "bf16", 32, interleaved=True),
        # one request answering: a single token over a short context
        attend("attn_token", 1, 1, 0, 4096, False, 40, 8, 128, "fp8", 16),
        # a decode step of 64 requests of uneven lengths
        attend("attn_decode", 64, 1, 0, 32768, True, 40, 8, 128, "fp8", 16),
        # a few drafted tokens of each request checked at once, bf16 cache, narrow heads
        attend("attn_drafts_bf16", 16, 4, 16, 8191, True, 32, 8, 64, "bf16", 16, lse=True),
        # a chunk of a long prompt over what the cache holds already
        attend("attn_chunk", 1, 512, 1, 32768, False, 40, 8, 128, "fp8", 64),
        # a whole prompt at once
        attend("attn_prefill", 1, 8192, 1, 8192, False, 40, 8, 128, "fp8", 64),
        # prompt chunks beside single tokens, wide heads, sliding window
        attend("attn_mixed_window", 17, 300, 4, 6000, True, 16, 2, 256, "bf16", 32, window=2048, lse=True),
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention"])
    q_heads, kv_heads = rng.choice([(40, 8), (32, 8), (16, 2), (24, 4), (8, 8), (20, 4), (28, 4)])
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    cache = rng.choice(["fp8", "fp8", "bf16"])
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "norm_rope":
        return {"op": op, "tokens": _between(rng, 1, 8192), "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "norm": rng.random() < 0.8, "interleaved": rng.random() < 0.3}
    seqs = _between(rng, 1, 64)
    chunks = rng.choice([0, 0, 1, seqs])
    if op == "append":
        new = 1 if chunks == 0 else _between(rng, 2, max(2, 8192 // chunks))
        kv = new + _between(rng, 1, 8192)
        return {"op": op, "seqs": seqs, "new": new, "chunks": chunks, "kv": kv, "ragged": rng.random() < 0.6,
                "q_heads": rng.choice([0, q_heads, q_heads]), "kv_heads": kv_heads, "dim": dim, "rot": rot, "cache": cache,
                "page": page, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), "interleaved": rng.random() < 0.3}
    new = 1 if chunks == 0 else _between(rng, 2, max(2, 4096 // chunks))
    # pairs of queries and keys and bytes of cache stay below the largest listed case's
    most = min(2 ** 25 // (seqs * kv_heads) * 128 // dim, 2 ** 25 // ((chunks * new + seqs) * q_heads) * 16, 32768)
    kv = max(new, _between(rng, 16, max(17, most)))
    return {"op": op, "seqs": seqs, "new": new, "chunks": chunks, "kv": kv, "ragged": rng.random() < 0.6, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page, "window": rng.choice([0, 0, 0, 128, 1000]),
            "causal": rng.random() < 0.9, "lse": rng.random() < 0.3}


def _lengths(case):
    """New tokens and cache lengths of every sequence; the same for every seed."""
    S = case["seqs"]
    new = [case["new"] if i < case["chunks"] else 1 for i in range(S)]
    kv = [case["kv"] if not case["ragged"] else case["kv"] * ((i * 29) % S + 1) // S for i in range(S)]
    return new, [max(a, b) for a, b in zip(new, kv)]


def _window(case):
    return case["window"] if case["causal"] else 0


def _pairs(case):
    """Queries times the keys each one sees, and the cache rows any query of a sequence sees."""
    pairs = rows = 0
    for n, L in zip(*_lengths(case)):
        w = _window(case) or L
        if not case["causal"]:
            pairs, rows = pairs + n * L, rows + L
            continue
        # query i of n sees min(L - n + i + 1, w) keys
        short = max(0, min(n, w - (L - n)))           # queries that see every key before them
        pairs += short * (L - n) + short * (short + 1) // 2 + (n - short) * w
        rows += min(L, w + n - 1)
    return pairs, rows


def work(case):
    D = case["dim"]
    if case["op"] == "norm_rope":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * D
        return {"bytes": 2 * n * e + case["tokens"] * (case["rot"] * 4 + 8), "flops": n * 8}
    new, kv = _lengths(case)
    c = 1 if case["cache"] == "fp8" else 2
    T = sum(new)
    if case["op"] == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        q, k = T * case["q_heads"] * D, T * case["kv_heads"] * D
        return {"bytes": 2 * q * e + 2 * k * (e + c) + T * case["rot"] * 4, "flops": 8 * (q + 2 * k)}
    pairs, rows = _pairs(case)
    return {"bytes": 2 * rows * case["kv_heads"] * D * c + 4 * T * case["q_heads"] * D + 4 * T * case["q_heads"] * case["lse"],
            "flops": 4 * pairs * case["q_heads"] * D}


def _draw_of(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(1_000_003 * int(seed) + 17)


def _table(positions, rot):
    """cos | sin of every position's angles, from 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g = _draw_of(seed)
    D, Hq, Hk = case["dim"], case["q_heads"], case["kv_heads"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "norm_rope":
        T, dt = case["tokens"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # queries and keys are column ranges of one fused projection's output
        qkv = (randn(T, (Hq + 2 * Hk) * D) * 1.5).to(dt)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        s["q_weight"] = 1 + 0.2 * randn(D) if case["norm"] else None
        s["k_weight"] = 1 + 0.2 * randn(D) if case["norm"] else None
        s["rope"] = _table(16384, case["rot"])
        s["positions"] = torch.randint(0, 16384, (T,), generator=g, device="cuda", dtype=torch.int32)
        return s
    new, kv = _lengths(case)
    page, S, T = case["page"], case["seqs"], sum(new)
    blocks = [-(-n // page) for n in kv]
    pages = sum(blocks) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(S, max(blocks), dtype=torch.int32)
    at = torch.zeros(S, max(blocks), dtype=torch.bool)
    for i, b in enumerate(blocks):
        at[i, :b] = True
    s["page_table"] = table.cuda().masked_scatter_(at.cuda(), order)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    s["max_q"], s["max_kv"] = max(new), max(kv)
    # keys with uneven channels, as after a trained norm; calibrated scales max|x| / 448
    gain = torch.linspace(0.2, 2.0, D, device="cuda")
    shape = (pages, Hk, page, D)
    fp8 = case["cache"] == "fp8"
    s["k_scale"] = torch.full((1,), 9.0 / 448, device="cuda") if fp8 else None
    s["v_scale"] = torch.full((1,), 6.0 / 448, device="cuda") if fp8 else None

    def cached(x, scale):
        if not fp8:
            return x.to(torch.bfloat16)
        return (x / scale).clamp_(-448, 448).to(E4M3).view(torch.uint8)

    if case["op"] == "attention":
        s["k_cache"] = cached(randn(*shape).mul_(gain), s["k_scale"])
        s["v_cache"] = cached(randn(*shape), s["v_scale"])
        s["q"] = randn(T, Hq, D).mul_(1.5).to(torch.bfloat16)
        return s
    s["k_cache"] = torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = (randn(T, (Hq + 2 * Hk) * D) * 1.2).to(dt)
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else None
    s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    s["v"] = qkv[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
    s["q_weight"] = 1 + 0.2 * randn(D) if Hq else None
    s["k_weight"] = 1 + 0.2 * randn(D)
    s["rope"] = _table(s["max_kv"], case["rot"])
    return s


def _normed(x, w, eps=1e-6):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _rotated(x, row, interleaved):
    """The first row.shape[-1] channels of x [T, H, D] rotated by the angles of row = cos | sin [T, R]."""
    R = row.shape[-1]
    c, n = row[:, None, :R // 2], row[:, None, R // 2:]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        r = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        r = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([r, x[..., R:]], -1)


def _plain_norm_rope(s):
    case, row = s["case"], s["rope"][s["positions"].long()]
    return [_rotated(_normed(s[n], s[n + "_weight"]), row, case["interleaved"]).to(s[n].dtype) for n in ("q", "k")]


def _plain_append(s):
    case, cu, kv_len = s["case"], s["cu_q"].long(), s["kv_len"].long()
    t = torch.arange(s["k"].shape[0], device="cuda")
    seq = (cu[None, :] <= t[:, None]).sum(1) - 1
    pos = kv_len[seq] - (cu[seq + 1] - t)
    row = s["rope"][pos]
    pg = s["page_table"][seq, pos // case["page"]].long()
    off = pos % case["page"]
    for cache, x, scale in ((s["k_cache"], _rotated(_normed(s["k"], s["k_weight"]), row, case["interleaved"]), s["k_scale"]),
                            (s["v_cache"], s["v"].float(), s["v_scale"])):
        cache[pg, :, off] = x.to(torch.bfloat16) if scale is None else (x / scale).clamp(-448, 448).to(E4M3).view(torch.uint8)
    q = None
    if s["q"] is not None:
        q = _rotated(_normed(s["q"], s["q_weight"]), row, case["interleaved"]).to(torch.bfloat16)
    return q


def _plain_attention(s):
    case, cu, kv_len = s["case"], s["cu_q"].long(), s["kv_len"].long()
    S, Hk, D, G, N, L = case["seqs"], case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"], s["max_q"], s["max_kv"]

    def gathered(cache, scale):
        x = cache[s["page_table"].long()]                                   # [S, blocks, Hk, page, D]
        x = x.transpose(1, 2).reshape(S, Hk, -1, D)[:, :, :L]
        return x.float() if scale is None else x.view(E4M3).float() * scale

    i = torch.arange(N, device="cuda")
    new = cu[1:] - cu[:-1]
    there = i[None, :] < new[:, None]                                        # [S, N]
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().unflatten(2, (Hk, G)).permute(0, 2, 1, 3, 4).reshape(S, Hk, N * G, D)
    p = q @ gathered(s["k_cache"], s["k_scale"]).transpose(2, 3).contiguous()
    p *= D ** -0.5
    pos = (kv_len - new)[:, None] + i                                        # [S, N]
    key = torch.arange(L, device="cuda")
    seen = (key < kv_len[:, None, None]).expand(S, N, L)
    if case["causal"]:
        seen = seen & (key <= pos[:, :, None])
        if case["window"]:
            seen = seen & (key > pos[:, :, None] - case["window"])
    p = p.view(S, Hk, N, G, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(S, Hk, N * G, L) @ gathered(s["v_cache"], s["v_scale"])).view(S, Hk, N, G, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 2, 1, 3, 4).flatten(2, 3)[there]
    lse = (m + l.log())[..., 0].permute(0, 2, 1, 3).flatten(2, 3)[there]
    return o.to(torch.bfloat16), lse


def run(s):
    case = s["case"]
    if own:
        import nvfp4_w4a4_block_amd as nv
    if case["op"] == "norm_rope":
        if own:
            return nv.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], rope=s["rope"], positions=s["positions"],
                                   interleaved=case["interleaved"])
        return _plain_norm_rope(s)
    if own:
        kv = nv.PagedKV(s["k_cache"], s["v_cache"], s["page_table"], s["k_scale"], s["v_scale"])
    if case["op"] == "append":
        if own:
            q = nv.kv_append(kv, s["k"], s["v"], s["kv_len"], s["cu_q"], k_weight=s["k_weight"], rope=s["rope"], q=s["q"],
                             q_weight=s["q_weight"], interleaved=case["interleaved"])
        else:
            q = _plain_append(s)
        k, v = s["k_cache"], s["v_cache"]
        if case["cache"] == "fp8":          # the bytes as the values they stand for, in units of the calibrated scale
            k, v = k.view(E4M3), v.view(E4M3)
        return [k, v] if q is None else [k, v, q]
    if own:
        out = nv.paged_attention(s["q"], kv, s["kv_len"], s["cu_q"], causal=case["causal"], window=_window(case),
                                 max_q=s["max_q"], return_lse=case["lse"])
        return out
    o, lse = _plain_attention(s)
    return (o, lse) if case["lse"] else o


def _e4m3_64(x):
    """Nearest E4M3 value of 64-bit numbers: three mantissa bits, spacing 2^-9 below 2^-6, at most 448; ties to even."""
    a = x.abs().clamp(max=448.0)
    e = torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 4
    step = torch.ldexp(torch.ones_like(a), e)
    return torch.copysign((a / step).round() * step, x)


def _turn_64(x, w, positions, rot, interleaved):
    """Norm and rotation in 64 bits with complex numbers: channel pairs times the table's cos + i sin."""
    z = x.double()
    if w is not None:
        z = z * w.double() / ((z.square().sum(-1, keepdim=True) / z.shape[-1]) + 1e-6).sqrt()
    table = _table(int(positions.max()) + 1, rot)[positions.long()].double()
    unit = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]
    head = z[..., :rot]
    pair = head.unflatten(-1, (rot // 2, 2)) if interleaved else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
    turned = turned if interleaved else turned.transpose(-1, -2)
    return torch.cat([turned.reshape(head.shape), z[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return [_turn_64(s[n], s[n + "_weight"], s["positions"], case["rot"], case["interleaved"]) for n in ("q", "k")]
    new, kv = _lengths(case)
    page, Hk, D = case["page"], case["kv_heads"], case["dim"]
    table = s["page_table"].long()
    if case["op"] == "append":
        positions = torch.cat([torch.arange(L - n, L) for n, L in zip(new, kv)]).cuda()
        k = _turn_64(s["k"], s["k_weight"], positions, case["rot"], case["interleaved"])
        caches, start = [torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda") for _ in range(2)], 0
        for i, (n, L) in enumerate(zip(new, kv)):
            p = positions[start:start + n]
            for cache, x, scale in ((caches[0], k, s["k_scale"]), (caches[1], s["v"].double(), s["v_scale"])):
                y = x[start:start + n]
                cache[table[i, p // page], :, p % page] = y if scale is None else _e4m3_64(y / scale.double())
            start += n
        q = [] if s["q"] is None else [_turn_64(s["q"], s["q_weight"], positions, case["rot"], case["interleaved"])]
        return caches + q
    G, start = case["q_heads"] // Hk, 0
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, (n, L) in enumerate(zip(new, kv)):
        key = torch.arange(L, device="cuda")
        at = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = (key > at) if case["causal"] else torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if _window(case):
            hidden = hidden | (key <= at - _window(case))
        for h in range(Hk):
            def rows(cache, scale):
                x = cache[table[i, :-(-L // page)], h].reshape(-1, D)[:L]
                return x.double() if scale is None else x.view(E4M3).double() * scale.double()
            K, V = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
            for j in range(h * G, (h + 1) * G):
                x = (s["q"][start:start + n, j].double() @ K.T) / math.sqrt(D)
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[start:start + n, j] = z
                o[start:start + n, j] = (x - z[:, None]).exp() @ V
        start += n
    return (o, lse) if case["lse"] else o

"""Cases of the operators between the 4-bit linears of a Gated DeltaNet layer: the residual's
addition with a root-mean-square norm and a quantized output (``add_rms_norm``), the causal
convolution with its state (``gdn_conv``), the gated delta rule over a batch of sequences
(``gated_delta_rule``) and the gated norm behind it (``gated_rms_norm``), in a plain form of
elementary torch operations and as the library's calls.

A case is a dict of plain values: ``op`` and the sizes it needs.  A batch of ``seqs`` sequences
has ``new`` new tokens in each of its first ``chunks`` sequences and one in every other one, after
``past`` tokens (0: every sequence starts here).  Head counts follow the fused input projection of
the benchmark's model (2048 / 2048 / 4096 / 4096 columns of queries, keys, values and output gates:
16 key heads and 32 value heads of 128) beside generic ones; rows of 5120 are its hidden size.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 2.0 ** -20


def listed():
    def norm(name, rows, cols, dtype, residual, quant, mode):
        return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "quant": quant,
                "mode": mode}

    def gated(name, rows, heads, dim, quant):
        return {"name": name, "op": "gated", "rows": rows, "heads": heads, "dim": dim, "quant": quant}

    def conv(name, seqs, new, chunks, past, k_heads, v_heads, dim, width, bias):
        return {"name": name, "op": "conv", "seqs": seqs, "new": new, "chunks": chunks, "past": past, "k_heads": k_heads,
                "v_heads": v_heads, "dim": dim, "width": width, "bias": bias}

    def delta(name, seqs, new, chunks, past, k_heads, v_heads, dim):
        return {"name": name, "op": "delta", "seqs": seqs, "new": new, "chunks": chunks, "past": past, "k_heads": k_heads,
                "v_heads": v_heads, "dim": dim}

    return [
        # one token in front of a linear, its NVFP4 scales by row: launch latency
        norm("norm_token", 1, 5120, "bf16", True, "nvfp4", "per_row"),
        # a prompt of the benchmark's length in front of a linear, calibrated scale
        norm("norm_prefill", 4096, 5120, "bf16", True, "nvfp4", "given"),
        # fp32 activations leaving as FP8 with a scale per row, an odd number of them, nothing to add
        norm("norm_fp8_f32", 2049, 4096, "f32", False, "fp8", "per_row"),
        # a decode step of 64 requests
        conv("conv_decode", 64, 1, 0, 4096, 16, 32, 128, 4, False),
        # a long prompt
        conv("conv_prefill", 1, 8192, 1, 0, 16, 32, 128, 4, False),
        # one request answering: a single token
        delta("delta_token", 1, 1, 0, 4096, 16, 32, 128),
        # a decode step of 64 requests: the states' bytes
        delta("delta_decode", 64, 1, 0, 4096, 16, 32, 128),
        # several prompts at once
        delta("delta_prompts", 8, 1023, 8, 0, 16, 32, 128),
        # a whole long prompt: the scan along the sequence
        delta("delta_prefill", 1, 8192, 1, 0, 16, 32, 128),
        # prompt chunks that go on beside single tokens, three value heads to a key head
        delta("delta_mixed", 17, 509, 5, 2048, 16, 48, 128),
        # a decode step's heads leaving as FP8 with a scale per token
        gated("gated_decode_fp8", 64, 32, 128, "fp8"),
        # a long prompt's heads
        gated("gated_prefill", 8192, 32, 128, "none"),
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gated", "conv", "delta", "delta", "delta"])
    if op == "norm":
        quant, cols = rng.choice(["nvfp4", "nvfp4", "fp8", "none"]), 16 * rng.choice([64, 128, 160, 255, 256, 320, 448, 512])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "rows": _between(rng, 1, 2 ** 24 // cols), "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.7, "quant": quant,
                "mode": "per_row" if quant == "none" else rng.choice(["per_row", "per_row", "given"])}
    k_heads, v_heads, dim = rng.choice([(16, 32, 128), (16, 48, 128), (8, 32, 128), (4, 8, 128), (16, 16, 128), (8, 32, 64), (2, 2, 64)])
    if op == "gated":
        return {"op": op, "rows": _between(rng, 1, 2 ** 25 // (v_heads * dim)), "heads": v_heads, "dim": dim,
                "quant": rng.choice(["fp8", "none"])}
    seqs = _between(rng, 1, 64)
    chunks = rng.choice([0, 1, seqs, seqs])
    new = 1 if chunks == 0 else _between(rng, 2, max(2, 2 ** 18 // (chunks * max(v_heads, 32))))
    case = {"op": op, "seqs": seqs, "new": new, "chunks": chunks, "past": rng.choice([0, 1, 2, 1000, 4096]), "k_heads": k_heads,
            "v_heads": v_heads, "dim": dim}
    if op == "conv":
        case |= {"width": rng.choice([4, 4, 3, 2]), "bias": rng.random() < 0.5}
    return case


def _new(case):
    return [case["new"] if i < case["chunks"] else 1 for i in range(case["seqs"])]


def work(case):
    if case["op"] == "norm":
        n, e = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        out = {"nvfp4": 9 / 16, "fp8": 1, "none": 2}[case["quant"]]
        return {"bytes": n * (e + (2 * e if case["residual"] else 0) + out) + 4 * case["cols"], "flops": 6 * n}
    if case["op"] == "gated":
        n = case["rows"] * case["heads"] * case["dim"]
        return {"bytes": n * (4 + (1 if case["quant"] == "fp8" else 2)), "flops": 10 * n}
    T, S, D = sum(_new(case)), case["seqs"], case["dim"]
    if case["op"] == "conv":
        C = (2 * case["k_heads"] + case["v_heads"]) * D
        old = S if case["past"] else 0
        return {"bytes": 4 * T * C + 2 * (S + old) * (case["width"] - 1) * C, "flops": T * C * (2 * case["width"] + 4)}
    Hk, Hv = case["k_heads"], case["v_heads"]
    old = S if case["past"] else 0
    return {"bytes": T * (4 * Hk * D + 4 * Hv * D + 8 * Hv) + 4 * (S + old) * Hv * D * D, "flops": 7 * T * Hv * D * D}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * int(seed) + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "norm":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows, cols = case["rows"], case["cols"]
        # a residual stream with a few channels far above the others
        gain = torch.ones(cols, device="cuda")
        gain[torch.randint(0, cols, (cols // 512,), generator=g, device="cuda")] = 40.0
        s["x"] = randn(rows, cols).to(dt)
        s["residual"] = (2 * randn(rows, cols) * gain).to(dt) if case["residual"] else None
        s["weight"] = 0.5 + rand(cols)
        s["scale"] = torch.full((1,), 0.02, device="cuda") if case["mode"] == "given" else None
        return s
    if case["op"] == "gated":
        T, H, D = case["rows"], case["heads"], case["dim"]
        s["x"] = (0.3 * randn(T, H, D)).to(torch.bfloat16)
        # the output gates are the projection's columns behind queries, keys and values
        s["z"] = randn(T, 3 * H * D).to(torch.bfloat16)[:, 2 * H * D:].unflatten(1, (H, D))
        s["weight"] = 0.5 + rand(D)
        return s
    new = _new(case)
    S, T, D, Hk, Hv = case["seqs"], sum(new), case["dim"], case["k_heads"], case["v_heads"]
    s["cu_q"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    s["kv_len"] = torch.tensor([n + case["past"] for n in new], dtype=torch.int32, device="cuda")
    s["slots"] = torch.randperm(S + 2, generator=g, device="cuda")[:S].to(torch.int32)
    s["max_q"] = max(new)
    C = (2 * Hk + Hv) * D
    if case["op"] == "conv":
        W = case["width"]
        s["x"] = randn(T, C + Hv * D).to(torch.bfloat16)[:, :C]            # the projection's first columns
        s["weight"] = 0.5 * randn(C, W)
        s["bias"] = 0.1 * randn(C) if case["bias"] else None
        s["state"] = randn(S + 2, W - 1, C).to(torch.bfloat16)
        return s
    # what the convolution gives: silu of about normal values, queries, keys and values side by side
    x = randn(T, C)
    x = (x * torch.sigmoid(x)).to(torch.bfloat16)
    s["q"] = x[:, :Hk * D].unflatten(1, (Hk, D))
    s["k"] = x[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D))
    s["v"] = x[:, 2 * Hk * D:].unflatten(1, (Hv, D))
    # log decays from almost none to strong, by head
    a = randn(T, Hv) - 2.25 - 4.65 * rand(Hv)
    s["g"] = -torch.exp(2.77 * rand(Hv)) * torch.log1p(torch.exp(a))
    s["beta"] = torch.sigmoid(randn(T, Hv))
    s["state"] = 0.2 * randn(S + 2, Hv, D, D)
    return s


def _e4m3(t):
    """Bytes of the E4M3 values nearest to t, at most 448."""
    return t.clamp(-448, 448).to(E4M3)


def _divided(x, d):
    """fl32(x / d) of 32-bit numbers: the quotient in 64 bits rounds to the same."""
    return (x.double() / d.double()).float()


def _nvfp4(y, mode, given):
    """Codes, scale bytes and global scale of 32-bit rows y, step by step in 32 bits as the format has it."""
    rows, cols = y.shape
    top = y.abs().amax(1)
    G = given if mode == "given" else _divided(top, torch.full_like(top, 2688.0))
    blocks = y.view(rows, cols // 16, 16)
    den = (6.0 * G)[:, None].expand(rows, cols // 16)
    scale = torch.where(den > 0, _e4m3(_divided(blocks.abs().amax(2), den)).float(), 0.0)
    d = (scale * G[:, None])[..., None]
    t = torch.where(d > 0, _divided(blocks.abs(), d.expand_as(blocks)), 0.0)
    # the eight magnitudes' midpoints; a tie goes to the even code
    idx = (t > 0.25).int() + (t >= 0.75).int() + (t > 1.25).int() + (t >= 1.75).int() + (t > 2.5).int() + (t >= 3.5).int() + (t > 5.0).int()
    code = (idx + 8 * torch.signbit(blocks).int()).view(rows, cols // 2, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), scale.to(E4M3).view(torch.uint8), G


def _plain_out(y, case, given=None):
    """The outputs of 32-bit rows y."""
    if case["quant"] == "none":
        return [y.to(torch.bfloat16)]
    if case["quant"] == "nvfp4":
        return list(_nvfp4(y, case["mode"], given))
    top = y.abs().amax(1)
    G = given if given is not None else _divided(top, torch.full_like(top, 448.0))
    return [_e4m3(_divided(y, G[:, None].expand_as(y))), G]


def _plain_norm(s):
    case, out = s["case"], []
    x = s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
        out = [x]
    # in 64 bits: the codes of values next to a border go by the last bits
    x = x.double()
    inv = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    return out + _plain_out((x * s["weight"].double() * inv).float(), case, s["scale"])


def _plain_gated(s):
    x, z = s["x"].float(), s["z"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"] * (z * torch.sigmoid(z))
    return _plain_out(y.flatten(1), s["case"])


def _sequence_of(s):
    """Every new token's sequence and its number in it."""
    cu = s["cu_q"].long()
    t = torch.arange(sum(_new(s["case"])), device="cuda")
    seq = (cu[None, :] <= t[:, None]).sum(1) - 1
    return t, seq, t - cu[seq]


def _plain_conv(s):
    case, W, x = s["case"], s["case"]["width"], s["x"]
    t, seq, i = _sequence_of(s)
    slots, n = s["slots"].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    old = s["state"][slots].float() * (s["kv_len"] > n)[:, None, None]
    back = torch.arange(W, device="cuda") - (W - 1)                         # -(W-1) .. 0
    at = i[:, None] + back                                                  # [T, W], negative: in the state
    taps = torch.where(at[..., None] >= 0, x[(t[:, None] + back).clamp(min=0)].float(), old[seq[:, None], (at + W - 1).clamp(0, W - 2)])
    y = (taps * s["weight"].T).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    last = n[:, None] + back[1:] - 1                                        # the state keeps inputs n-W+1 .. n-1
    first = s["cu_q"][:-1].long()[:, None]
    kept = torch.where(last[..., None] >= 0, x[(first + last).clamp(0, x.shape[0] - 1)].float(),
                       old[torch.arange(len(n), device="cuda")[:, None], (last + W - 1).clamp(0, W - 2)])
    s["state"][slots] = kept.to(torch.bfloat16)
    return (y * torch.sigmoid(y)).to(torch.bfloat16)


def _plain_delta(s):
    case, C = s["case"], 64
    S, Hv, D, G = case["seqs"], case["v_heads"], case["dim"], case["v_heads"] // case["k_heads"]
    _, seq, i = _sequence_of(s)
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    if s["max_q"] == 1:
        C = 1
    B = -(-s["max_q"] // C)

    def padded(x):
        """[T, H, ...] as [S, Hv, blocks, C, ...], zeros behind each sequence's end."""
        x = x.float() if x.shape[1] == Hv else x.float().repeat_interleave(G, 1)
        p = x.new_zeros((S, B * C) + x.shape[1:])
        p[seq, i] = x
        return p.transpose(1, 2).unflatten(2, (B, C))

    q, k, v, g, beta = (padded(s[name]) for name in ("q", "k", "v", "g", "beta"))
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6) * D ** -0.5
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    sums = g.double().cumsum(3)                                             # log decays since the block's start
    decay = torch.exp((sums[..., :, None] - sums[..., None, :]).clamp(max=0)).float()
    low = torch.ones(C, C, device="cuda").tril()
    A = (q @ k.transpose(-1, -2).contiguous()) * decay * low
    L = ((k @ k.transpose(-1, -2).contiguous()) * decay * beta[..., None] * low.tril(-1)).double()
    # (1 + L)^-1 = (1 - L)(1 + L^2)(1 + L^4) ..., L^C = 0; in 64 bits, its terms cancel
    one, P = torch.eye(C, dtype=torch.float64, device="cuda"), L @ L
    inverse = one - L
    for _ in range(max(0, C.bit_length() - 2)):
        inverse, P = inverse + inverse @ P, P @ P
    inverse = inverse.float()
    since, until = torch.exp(sums).float(), torch.exp(sums[..., -1:] - sums).float()
    slots = s["slots"].long()
    state = s["state"][slots] * (s["kv_len"] > n)[:, None, None, None]
    out = torch.empty_like(v)
    for b in range(B):
        e, kb = since[:, :, b, :, None], k[:, :, b]
        u = inverse[:, :, b] @ (beta[:, :, b, :, None] * (v[:, :, b] - e * (kb @ state)))
        out[:, :, b] = e * (q[:, :, b] @ state) + A[:, :, b] @ u
        state = state * e[:, :, -1:] + (kb * until[:, :, b, :, None]).transpose(-1, -2).contiguous() @ u
    s["state"][slots] = state
    return out.flatten(2, 3).transpose(1, 2)[seq, i].to(torch.bfloat16)


def run(s):
    case = s["case"]
    if own:
        import nvfp4_w4a4_block_amd as nv
        if case["op"] == "norm":
            dt = torch.bfloat16 if case["quant"] == "none" else None
            y, t, r = nv.add_rms_norm(s["x"], s["weight"], s["residual"], EPS, dt, case["quant"], case["mode"], s["scale"])
        elif case["op"] == "gated":
            dt = torch.bfloat16 if case["quant"] == "none" else None
            y, t = nv.gated_rms_norm(s["x"], s["z"], s["weight"], EPS, dt, case["quant"])
            r = None
        elif case["op"] == "conv":
            state = nv.GDNState(s["slots"], conv=s["state"])
            return [nv.gdn_conv(state, s["x"], s["weight"], s["kv_len"], s["cu_q"], bias=s["bias"]), s["state"]]
        else:
            state = nv.GDNState(s["slots"], delta=s["state"])
            o = nv.gated_delta_rule(state, s["q"], s["k"], s["v"], s["g"], s["beta"], s["kv_len"], s["cu_q"], max_q=s["max_q"])
            return [o, s["state"]]
        out = [] if r is None else [r]
        if case["quant"] == "none":
            return out + [y]
        if case["quant"] == "fp8":
            return out + [t.codes.view(E4M3), t.scale]
        return out + [t.codes, t.scales, t.global_scale]
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "gated":
        return _plain_gated(s)
    if case["op"] == "conv":
        return [_plain_conv(s), s["state"]]
    return [_plain_delta(s), s["state"]]


def _exact_out(y, case, given):
    if case["quant"] == "none":
        return [y]
    if case["quant"] == "nvfp4":
        return [None, None, y.abs().amax(1) / 2688 if given is None else given.double()]
    G = y.abs().amax(1) / 448 if given is None else given.double()
    t = (y / G[:, None]).clamp(-448, 448)
    # nearest of the values with three bits behind the first, 2^-9 apart below 2^-6; ties to even
    step = torch.ldexp(torch.ones_like(t), torch.frexp(t.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return [(t / step).round() * step, G]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, out = s["x"].double(), []
        if s["residual"] is not None:
            total = x + s["residual"].double()
            out, x = [total], total.to(s["x"].dtype).double()
        root = (x.pow(2).sum(1, keepdim=True) / case["cols"] + EPS).sqrt()
        return out + _exact_out(x / root * s["weight"].double(), case, s["scale"])
    if case["op"] == "gated":
        x, z = s["x"].double(), s["z"].double()
        root = (x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
        return _exact_out((x / root * s["weight"].double() * z / (1 + (-z).exp())).flatten(1), case, None)
    new, slots = _new(case), s["slots"].tolist()
    if case["op"] == "conv":
        W, at, out, state = case["width"], 0, [], s["state"].double()
        for n, slot in zip(new, slots):
            x = torch.cat([state[slot] if case["past"] else torch.zeros_like(state[slot]), s["x"][at:at + n].double()])
            y = sum(x[j:j + n] * s["weight"][:, j].double() for j in range(W))
            y = y if s["bias"] is None else y + s["bias"].double()
            out.append(y / (1 + (-y).exp()))
            state[slot] = x[n:]
            at += n
        return [torch.cat(out), state]
    # token by token, the sequences of the same length together
    G, D = case["v_heads"] // case["k_heads"], case["dim"]
    q, k = (s[n].double() / (s[n].double().square().sum(-1, keepdim=True) + 1e-6).sqrt() for n in ("q", "k"))
    q, k = q.repeat_interleave(G, 1) / math.sqrt(D), k.repeat_interleave(G, 1)
    v, decay, beta = s["v"].double(), s["g"].double().exp(), s["beta"].double()
    state, out, first = s["state"].double(), torch.empty(s["v"].shape, dtype=torch.float64, device="cuda"), s["cu_q"].long()
    lots = [range(case["chunks"]), range(case["chunks"], case["seqs"])]
    for lot in lots:
        if not len(lot):
            continue
        rows = s["slots"].long()[lot.start:lot.stop]
        M = state[rows] if case["past"] else torch.zeros_like(state[rows])
        for i in range(new[lot.start]):
            t = first[lot.start:lot.stop] + i
            M = M * decay[t][..., None, None]
            u = beta[t][..., None] * (v[t] - (M * k[t][..., None]).sum(2))
            M = M + k[t][..., None] * u[..., None, :]
            out[t] = (M * q[t][..., None]).sum(2)
        state[rows] = M
    return [out, state]

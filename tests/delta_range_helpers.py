"""The gated delta rule token by token in 64 bits, with tolerances that count nothing but 32-bit arithmetic and the output's
rounding to bf16: those of ``gdn_helpers.delta_rule`` also allow single fp16 operands in the outputs."""
from __future__ import annotations

import torch

from tests.gdn_helpers import U, Seqs

BLOCK = 64


def exact_rule(b: Seqs, q, k, v, g, beta, state, scale=None):
    """(out, out's tolerance, states, states' tolerance); rows of nobody are NaN.

    B bounds a column's 2-norm, B <- e^g B + |beta v|, and one step is a contraction of S's columns, so errors made at one token
    never grow.  A token's sums have Dk terms, a block's form of 64 tokens 64 more, every operand is held to
    2^-21 or better: its error is at most u (|beta v| + 2 B), u = 4 sqrt(Dk + 128) 2^-24, four times what independent
    roundings of the largest size add up to; errors of several tokens are independent, E^2 <- e^2g E^2 + (that)^2.  The
    output's own sum, over Dk channels and up to 64 updates, makes another u B.
    Values far below what the same block of 64 holds are held to a part of that: two fp16 parts, the second scaled by 2^11, in
    units that take M, the block's bound, below 2^13 leave 2^-25 2^-11 2^-12 M = 2^-48 M an element, a sum of at most 64 of them
    (|T_ij| <= 2) 2^-41 M at most.  M is at most the columns' 1-norm (sqrt(Dk) B) and 64 |beta v| a block: 80 P for P the largest
    B of the last 128 tokens and two blocks (twice 64 of beta v, sqrt(128) of B), 2^8 P with its slack: 2^-33 P."""
    T, Hv, Dv = v.shape
    Dk, G = q.shape[2], Hv // q.shape[1]
    scale = Dk ** -0.5 if scale is None else scale

    def unit(x):
        x = x.double()
        return (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(G, 1)

    qn, kn, vd, gd, bd = unit(q), unit(k), v.double(), g.double(), beta.double()
    out = torch.full((T, Hv, Dv), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    states, tols = state.double().clone(), torch.zeros(state.shape, dtype=torch.float64)
    u32 = 4 * (Dk + 2 * BLOCK) ** 0.5 * U
    for i, (f, n) in enumerate(zip(b.first, b.new)):
        if n == 0:
            continue
        slot = b.slot(i)
        S = states[slot].clone() if slot is not None and b.past[i] > 0 else torch.zeros((Hv, Dk, Dv), dtype=torch.float64)
        B = S.square().sum(1).sqrt()
        E, seen = torch.zeros_like(B), [B]
        for t in range(f, f + n):
            e = gd[t].exp()[:, None]
            S = S * e[..., None]
            u = bd[t][:, None] * (vd[t] - torch.einsum("hkv,hk->hv", S, kn[t]))
            S = S + kn[t][..., None] * u[:, None, :]
            out[t] = scale * torch.einsum("hkv,hk->hv", S, qn[t])
            written = bd[t][:, None].abs() * vd[t].abs()
            B = e * B + written
            E = torch.sqrt((e * E) ** 2 + (u32 * (written + 2 * B)) ** 2)
            seen = seen[-2 * BLOCK:] + [B]
            floor = 2.0 ** -33 * torch.stack(seen).amax(0)
            tol[t] = 2.0 ** -8 * out[t].abs() + scale * (E + u32 * B + floor) + 2.0 ** -120
        if slot is not None:
            states[slot] = S
            tols[slot] = (E + floor)[:, None, :].expand_as(S) + 2.0 ** -23 * S.abs() + 2.0 ** -120
    return out, tol, states, tols

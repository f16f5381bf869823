"""Plain 64-bit implementations of the paged-cache operators and the batches the tests run them on.

Tolerances are derived, per element, from the formulas (u = 2^-24 is half a step of fp32 relative to the
value, a rounding to bf16 at most 2^-8, to fp16 2^-11 relative or 2^-25 absolute).

Attention, row with exact scores s_j (natural exponent), probabilities p_j, n keys seen:
  * products of bf16 operands are exact in fp32, their sum over D channels is off by at most D u sum|q k|,
    the factor and the subtraction of the maximum by a few u of |s| and |max|: e = (D + 8) u S, S the
    largest scale * sum|q k| over the keys seen; the exponential adds 4 u;
  * each p_j is thus off by r = e + 2^-21 relative, twice that next to the normalised sum, whose own
    summation in fp32 adds n u; the rounding of p_j for the product with V adds 2^-11 relative
    and 2^-25 absolute (E4M3 cache; the row's sum is at least 1 in the scale of the rounded
    values) or 2^-8 relative (bf16 cache); the product's sum adds n u:
      |out - o| <= sum_j p_j |v_j| (2 r + 2 n u + P) + 2^-25 sum_j |v_j| + 2^-8 |o| (bf16 output);
  * lse: r + n u + 8 u |lse|.

Norm and rotation: sum of D squares in fp32 and root, quotient, products: at most (D / 8 + 16) u
relative on the normed value; the rotation's two products and their sum 3 u of |a cos| + |b sin|."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.gpu_helpers import DEV, nv

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def decode(cache: torch.Tensor) -> torch.Tensor:
    """Cache elements as float64 (E4M3 bytes or bf16)."""
    return (cache.view(E4M3).float() if cache.dtype == torch.uint8 else cache.float()).double()


class Batch:
    """A paged cache with random pages and a batch of sequences over it, on the CPU.

    new, kv: new tokens and cache lengths per sequence; lead / tail: rows of q before the first and behind
    the last sequence that belong to nobody; spare pages hold stale bytes, NaN patterns among them."""

    def __init__(self, new, kv, Hq, Hk, D, fp8=True, page=16, seed=0, lead=0, tail=0, width=None, spare=2, joint=False,
                 per_head=False, v_gain=1.0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.Hq, self.Hk, self.D, self.fp8, self.page = list(new), list(kv), Hq, Hk, D, fp8, page
        S = len(new)
        blocks = [-(-max(n, 0) // page) for n in kv]
        self.width = max(blocks + [1]) if width is None else width
        P = sum(blocks) + spare
        shape = (P, 2, Hk, page, D)
        x = torch.randn(shape, generator=g) * torch.linspace(0.3, 1.8, D)
        x[:, 1] *= v_gain
        if fp8:
            store = (x * 40).clamp(-448, 448).to(E4M3).view(torch.uint8)
            stale = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
            stale[..., ::7] = 0x7F
        else:
            store = x.to(torch.bfloat16)
            stale = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            stale[..., 1::3] = float("inf")
        order = torch.randperm(P, generator=g)
        self.table = torch.full((S, self.width), -7, dtype=torch.int32)
        used, at = torch.zeros(P, page, dtype=torch.bool), 0
        for s, b in enumerate(blocks):
            self.table[s, :b] = order[at:at + b].to(torch.int32)
            for j in range(b):
                used[order[at + j], :min(page, kv[s] - j * page)] = True
            at += b
        mask = used[:, None, None, :, None].expand(shape)
        both = torch.where(mask, store, stale)
        self.both = both if joint else None
        self.k, self.v = (both[:, 0], both[:, 1]) if joint else (both[:, 0].contiguous(), both[:, 1].contiguous())
        n = Hk if per_head else 1
        self.ks = 1 / 40 * torch.linspace(1.0, 1.5, n) if fp8 else None
        self.vs = 1 / 40 * torch.linspace(0.8, 1.4, n) if fp8 else None
        self.T = lead + sum(new) + tail
        cu = np.cumsum([lead] + list(new))
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.kv_len = torch.tensor(kv, dtype=torch.int32)
        self.q = (torch.randn(self.T, Hq, D, generator=g) * 1.3).to(torch.bfloat16)

    def device(self, dev=DEV):
        """(PagedKV, kv_len, cu_q, q) on the GPU."""
        if self.both is not None:
            both = self.both.to(dev)
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = self.k.to(dev), self.v.to(dev)
        f = lambda x: None if x is None else x.to(dev)  # noqa: E731
        return nv().PagedKV(k, v, self.table.to(dev), f(self.ks), f(self.vs)), self.kv_len.to(dev), self.cu.to(dev), self.q.to(dev)

    def scales(self, h):
        if not self.fp8:
            return 1.0, 1.0
        i = h if self.ks.numel() > 1 else 0
        return float(self.ks[i]), float(self.vs[i])

    def attention(self, scale=None, causal=True, window=0):
        """(out, lse, tolerance of out, tolerance of lse) in float64; rows of nobody are NaN in out."""
        D, G = self.D, self.Hq // self.Hk
        scale = D ** -0.5 if scale is None else scale
        out = torch.full((self.T, self.Hq, D), math.nan, dtype=torch.float64)
        lse = torch.full((self.T, self.Hq), math.nan, dtype=torch.float64)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        P = 2.0 ** -11 if self.fp8 else 2.0 ** -8
        for s, (n, L) in enumerate(zip(self.new, self.kv)):
            L = max(0, min(L, self.width * self.page))
            c0 = int(self.cu[s])
            pages = self.table[s, :-(-L // self.page)].long()
            ok = ((pages >= 0) & (pages < self.k.shape[0])).repeat_interleave(self.page)[:L]
            key, pos = torch.arange(L), (L - n + torch.arange(n))[:, None]
            seen = ok.expand(n, L).clone()
            if causal:
                seen &= key <= pos
                if window:
                    seen &= key > pos - window
            for h in range(self.Hk):
                ks, vs = self.scales(h)
                at = pages.clamp(0, self.k.shape[0] - 1)
                K = decode(self.k[at, h]).reshape(-1, D)[:L] * ks
                V = decode(self.v[at, h]).reshape(-1, D)[:L] * vs
                K = torch.where(ok[:, None], K, 0.0)
                bad = ~torch.isfinite(V) & ok[:, None]
                V0 = torch.where(torch.isfinite(V), V, 0.0)
                for j in range(h * G, (h + 1) * G):
                    q = self.q[c0:c0 + n, j].double()
                    x = (q @ K.T) * scale
                    x = torch.where(seen, x, -math.inf)
                    z = torch.logsumexp(x, -1) if L else torch.full((n,), -math.inf, dtype=torch.float64)
                    p = torch.where(seen, (x - torch.where(torch.isinf(z), 0.0, z)[:, None]).exp(), 0.0)
                    o = p @ V0
                    if bad.any():
                        up = (seen[:, :, None] & bad & ~(V == -math.inf)).any(1)
                        down = (seen[:, :, None] & bad & ~(V == math.inf)).any(1)
                        o = o + torch.where(up, math.inf, 0.0) + torch.where(down, -math.inf, 0.0)
                    out[c0:c0 + n, j], lse[c0:c0 + n, j] = o, z
                    cnt = seen.sum(1)[:, None].double()
                    S = torch.where(seen, (q.abs() @ K.nan_to_num().abs().T) * scale, 0.0).amax(-1, keepdim=True) if L else 0.0
                    r = (D + 8) * U * S + 2.0 ** -21
                    t = (p @ V0.abs()) * (2 * r + 2 * cnt * U + P) + 2.0 ** -8 * o.abs() + 1e-30
                    if self.fp8:
                        t = t + 2.0 ** -25 * (seen.double() @ V0.abs())
                    tol[c0:c0 + n, j] = t
                    tol_lse[c0:c0 + n, j] = (r + cnt * U)[:, 0] + 8 * U * z.abs()
        return out, lse, tol, tol_lse


def assert_close(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what: str = "") -> None:
    """|got - want| <= tol, infinities and NaNs equal; NaN in `want` of rows that belong to nobody has tol 0."""
    got = got.double().cpu()
    fine = torch.isfinite(want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    ok = torch.where(fine, (got - want).abs() <= tol, same)
    bad = torch.nonzero(~ok)
    assert bad.numel() == 0, (f"{what}: {len(bad)} of {want.numel()} out of tolerance, first {bad[0].tolist()}: got "
                              f"{got[tuple(bad[0])].item()} want {want[tuple(bad[0])].item()} tol {tol[tuple(bad[0])].item()}")


def rope_table(rows: int, rot: int, base: float = 10000.0) -> torch.Tensor:
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def norm_rope(x: torch.Tensor, w, table, pos, interleaved: bool, eps: float = 1e-6):
    """(y, tolerance of the fp32 value) in float64 of x [T, H, D]; pos: one per token, outside the table NaN."""
    z = x.double()
    D = x.shape[-1]
    rel = 0.0
    if w is not None:
        z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        rel = (D / 8 + 16) * U
    tol = z.abs() * rel
    if table is None:
        return z, tol
    R = table.shape[1]
    pos = torch.as_tensor(pos).long()
    known = (pos >= 0) & (pos < table.shape[0])
    row = torch.where(known[:, None], table[pos.clamp(0, max(0, table.shape[0] - 1))].double(), math.nan)[:, None]
    c, n = row[..., :R // 2], row[..., R // 2:]
    ia, ib = (torch.arange(0, R, 2), torch.arange(1, R, 2)) if interleaved else (torch.arange(R // 2), torch.arange(R // 2, R))
    a, b = z[..., ia], z[..., ib]
    y, t = z.clone(), tol.clone()
    y[..., ia], y[..., ib] = a * c - b * n, b * c + a * n
    e = (rel + 3 * U) * ((a * c).abs() + (b * n).abs()), (rel + 3 * U) * ((b * c).abs() + (a * n).abs())
    t[..., ia], t[..., ib] = e[0].nan_to_num(), e[1].nan_to_num()
    return y, t


def stored(y: torch.Tensor, tol: torch.Tensor, dtype) -> torch.Tensor:
    """Tolerance of the value y +- tol rounded to dtype (bf16, fp32)."""
    return tol + 1e-38 if dtype == torch.float32 else tol + 2.0 ** -8 * (y.abs() + tol) + 1e-38

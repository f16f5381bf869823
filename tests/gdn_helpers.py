"""Plain 64-bit implementations of the Gated DeltaNet layer's operators (norms with quantized outputs, causal
convolution, gated delta rule) and the tolerances of their tests, derived from the arithmetic."""
from __future__ import annotations

import numpy as np
import torch

from oracle import nvfp4_ref as ref
from tests.gpu_helpers import DEV, assert_quant_equal

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24                     # half a step of fp32, relative
HALF = {BF16: 2.0 ** -8, F32: U}   # half a step of an output type, relative


def rand(*shape, seed=0, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def uniform(*shape, seed=0):
    return torch.rand(*shape, generator=torch.Generator().manual_seed(seed))


def assert_within(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what: str = "") -> None:
    """|got - want| <= tol; NaN exactly where want is NaN, infinities equal."""
    g, w = got.detach().double().cpu(), want.double()
    assert g.shape == w.shape, what
    same = (g == w) | (torch.isnan(g) & torch.isnan(w))
    bad = ~(same | ((g - w).abs() <= tol))
    n = int(bad.sum())
    if n:
        at = tuple(int(i) for i in bad.nonzero()[0])
        assert False, f"{what}: {n} of {bad.numel()} out of tolerance, first {at}: got {g[at]}, want {w[at]}, tol {tol.expand_as(w)[at]}"


def silu(x: torch.Tensor) -> torch.Tensor:
    return x * torch.sigmoid(x)


# ---- norms ---------------------------------------------------------------------------------------


def add_norm64(x, residual, w, eps):
    """(r', y) of add_rms_norm, from the rounded sum on in 64 bits."""
    r = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    d = r.double()
    return r, d * w.double() * (1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + float(np.float32(eps))))


def add_norm(x, residual, w, eps):
    """(r', fl32(y))."""
    r, y = add_norm64(x, residual, w, eps)
    return r, y.float()


def check_quant(q, y: torch.Tensor, quant, mode, given):
    """The quantized output's bytes are those of y, 64 bits: NVFP4 as the oracle has it from fl32(y), FP8 the nearest."""
    if quant == "nvfp4":
        y = y.float().numpy()
        assert_quant_equal(q, ref.quantize(y, ref.PER_ROW) if mode == "per_row" else ref.quantize(y, ref.GIVEN, np.float32(given)))
        return
    y = y.double().numpy()
    scale = np.abs(y).max(1) / 448 if mode == "per_row" else np.full(len(y), np.float32(given), np.float64)
    if mode == "per_row":
        assert np.array_equal(q.scale.cpu().numpy(), scale.astype(np.float32))
    t = y / scale[:, None]
    assert np.array_equal(q.codes.cpu().numpy(), ref.e4m3_rne_sat(np.abs(t)) | np.where(np.signbit(t), 0x80, 0).astype(np.uint8))


def gated_norm(x, z, w, eps):
    """(y, tolerance without a quantized output, with one), before output rounding.  With one it is evaluated to 2^-40
    or better.  Without, roundings of the fp32 evaluation in units of U: the sum of squares 16 + 6 (a chain of 16, twice
    rounded, and a butterfly of at most six: 38), halved by the root: 19; mean, eps, root, quotient: 4; sigmoid: exponential
    2 + 2 |z| (its argument's rounding, twice where a constant is multiplied in), sum 1, quotient 1; products 3.
    Below 2^-100 the gate flushes."""
    d, g = x.double(), z.double()
    y = d / torch.sqrt((d * d).mean(-1, keepdim=True) + float(np.float32(eps))) * w.double() * silu(g)
    return y, U * (30 + 2 * g.abs()) * y.abs() + 2.0 ** -100, 2.0 ** -40 * y.abs() + 2.0 ** -126


# ---- sequences -----------------------------------------------------------------------------------


class Seqs:
    """A batch of sequences: new tokens and tokens held before, rows of nobody in front and behind, a pool of slots in
    a shuffled order."""

    def __init__(self, new, past, front=0, behind=0, spare=2, seed=0):
        self.new, self.past = list(new), list(past)
        self.first = [front + sum(self.new[:i]) for i in range(len(new))]
        self.T = front + sum(self.new) + behind
        g = torch.Generator().manual_seed(1000 + seed)
        self.num_slots = len(new) + spare
        self.slots = torch.randperm(self.num_slots, generator=g)[:len(new)].to(torch.int32)
        self.cu_q = torch.tensor(self.first + [front + sum(self.new)], dtype=torch.int32)
        self.kv_len = torch.tensor([n + p for n, p in zip(self.new, self.past)], dtype=torch.int32)

    def rows(self):
        m = torch.zeros(self.T, dtype=torch.bool)
        for f, n in zip(self.first, self.new):
            m[f:f + n] = True
        return m

    def gpu(self):
        return self.kv_len.to(DEV), self.cu_q.to(DEV)

    def slot(self, i):
        s = int(self.slots[i])
        return s if 0 <= s < self.num_slots else None


def conv(b: Seqs, x, weight, bias, state):
    """(y, tolerance before output rounding, new states): rows of nobody are NaN.  fp32: W + 1 roundings of the sum,
    through silu's slope (at most 1.1), and its own evaluation."""
    W = weight.shape[1]
    y = torch.full((b.T, x.shape[1]), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(y)
    state = state.clone()
    for i, (f, n) in enumerate(zip(b.first, b.new)):
        if n == 0:
            continue
        slot = b.slot(i)
        old = state[slot] if slot is not None and b.past[i] > 0 else torch.zeros((W - 1, x.shape[1]), dtype=x.dtype)
        seq = torch.cat([old, x[f:f + n]])
        d, w = seq.double(), weight.double()
        s = sum(d[j:j + n] * w[:, j] for j in range(W))
        a = sum((d[j:j + n] * w[:, j]).abs() for j in range(W))
        if bias is not None:
            s, a = s + bias.double(), a + bias.double().abs()
        y[f:f + n] = silu(s)
        tol[f:f + n] = 1.1 * (W + 1) * U * a + (8 + 2 * s.abs()) * U * silu(s).abs() + 2.0 ** -100
        if slot is not None:
            state[slot] = seq[n:]
    return y, tol, state


def delta_rule(b: Seqs, q, k, v, g, beta, state, scale=None):
    """(out, out's tolerance with its rounding to bf16, states, states' tolerance), token by token in 64 bits; rows of
    nobody are NaN.

    Tolerances.  One step is a contraction of S's columns (|k^| <= 1, 0 <= beta <= 2, g <= 0), so errors made at one
    token never grow.  B bounds a column's 2-norm: B <- e^g B + |beta v|.  One token's sums have Dk terms, a block's
    form of 64 tokens 64 more, every operand is held to 2^-21 or better: its error is at most
    4 sqrt(Dk + 64 + 64) U (|beta v| + 2 B), four times what independent roundings of the largest size add up to.
    Errors of several tokens are independent too, E^2 <- e^2g E^2 + (that)^2.
    An output reads S with q^, |q^| <= 1, and may take S and its products with single fp16 roundings: 2^-11 B, and
    2^-11 each for weights and updates of the tokens since: 2^-10 sum e^.. |u|."""
    T, Hv, Dv = v.shape
    Dk, G = q.shape[2], Hv // q.shape[1]
    scale = Dk ** -0.5 if scale is None else scale

    def unit(x):
        x = x.double()
        return (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(G, 1)

    qn, kn, vd, gd, bd = unit(q), unit(k), v.double(), g.double(), beta.double()
    out = torch.full((T, Hv, Dv), float("nan"), dtype=torch.float64)
    out_tol = torch.zeros_like(out)
    states, tols = state.double().clone(), torch.zeros(state.shape, dtype=torch.float64)
    unit_error = 4 * (Dk + 128) ** 0.5 * U
    for i, (f, n) in enumerate(zip(b.first, b.new)):
        if n == 0:
            continue
        slot = b.slot(i)
        S = states[slot].clone() if slot is not None and b.past[i] > 0 else torch.zeros((Hv, Dk, Dv), dtype=torch.float64)
        B = S.square().sum(1).sqrt()
        E, since = torch.zeros_like(B), torch.zeros_like(B)
        for t in range(f, f + n):
            e = gd[t].exp()[:, None]
            S = S * e[..., None]
            u = bd[t][:, None] * (vd[t] - torch.einsum("hkv,hk->hv", S, kn[t]))
            S = S + kn[t][..., None] * u[:, None, :]
            out[t] = scale * torch.einsum("hkv,hk->hv", S, qn[t])
            written = bd[t][:, None].abs() * vd[t].abs()
            B = e * B + written
            E = torch.sqrt((e * E) ** 2 + (unit_error * (written + 2 * B)) ** 2)
            since = e * since + u.abs()
            out_tol[t] = 2.0 ** -8 * out[t].abs() + scale * (E + 2.0 ** -11 * B + 2.0 ** -10 * since)
        if slot is not None:
            states[slot] = S
            tols[slot] = E[:, None, :].expand_as(S) + 2.0 ** -23 * S.abs()
    return out, out_tol, states, tols


def delta_inputs(b: Seqs, Hk, Hv, Dk, Dv, seed=0, strong=False):
    """What the convolution and the gates give: silu of normal values, side by side; decays from almost none to
    strong."""
    C = 2 * Hk * Dk + Hv * Dv
    x = silu(rand(b.T, C, seed=seed, dtype=F32)).to(BF16)
    q, k = x[:, :Hk * Dk].unflatten(1, (Hk, Dk)), x[:, Hk * Dk:2 * Hk * Dk].unflatten(1, (Hk, Dk))
    v = x[:, 2 * Hk * Dk:].unflatten(1, (Hv, Dv))
    a = rand(b.T, Hv, seed=seed + 1, dtype=F32) - 2.25 - 4.65 * uniform(Hv, seed=seed + 2)
    g = -torch.exp(2.77 * uniform(Hv, seed=seed + 3)) * torch.log1p(a.exp())
    if strong:
        g = g * 100
    beta = torch.sigmoid(rand(b.T, Hv, seed=seed + 4, dtype=F32))
    state = rand(b.num_slots, Hv, Dk, Dv, seed=seed + 5, dtype=F32, scale=0.2)
    return x, q, k, v, g, beta, state

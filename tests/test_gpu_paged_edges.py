"""Corners of the paged cache's operators against the plain 64-bit implementation: probabilities far below a row's
largest, scores of every size, non-finite values whatever the keys' division over wavefronts and workgroups."""
import math

import pytest
import torch

from tests.gpu_helpers import DEV, nv
from tests.paged_helpers import Batch, assert_close, decode

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def run(b: Batch, **kw):
    kv, kv_len, cu, q = b.device()
    out, lse = nv().paged_attention(q, kv, kv_len, cu, return_lse=True, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def place(b: Batch, s: int, key: int):
    """(page, row) of a key of sequence s."""
    return int(b.table[s, key // b.page]), key % b.page


def store(b: Batch, x: torch.Tensor) -> torch.Tensor:
    return x.to(torch.float8_e4m3fn).view(torch.uint8) if b.fp8 else x.to(BF16)


def one_channel_scores(b: Batch, scores: torch.Tensor) -> None:
    """Keys of sequence 0 whose score, before the scale, is scores[key] for every query: channel 0 of q is 1."""
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.k.zero_()
    if b.fp8:
        b.ks, b.vs = torch.ones(1), torch.ones(1)
    x = store(b, scores.float())
    for key in range(b.kv[0]):
        p, r = place(b, 0, key)
        b.k[p, :, r, 0] = x[key]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("n,L", [(1, 100), (1, 4000), (4, 700), (100, 900), (300, 4100)])
@pytest.mark.parametrize("below", [23.0, 25.5, 29.0])
def test_long_flat_tail_beside_a_peak(fp8, n, L, below):
    # key 0 has the row's largest score and a zero value, every other key a probability of 2^-below beside it, so
    # the output is what the small probabilities add up to.  Tolerance: a probability is held in a scale where the
    # row's sum is at least 2^7 next to fp16, whose absolute rounding is 2^-25: 2^-32 of |v| per key, not
    # the 2^-25 that a sum of 1 would leave.
    b = Batch([n], [L], 10, 2, 128, fp8, seed=n)
    scores = torch.zeros(L)
    scores[0] = 16.0
    one_channel_scores(b, scores)
    p0, r0 = place(b, 0, 0)
    b.v[p0, :, r0] = 0
    scale = below * math.log(2) / 16
    want, want_lse, tol, tol_lse = b.attention(scale)
    if fp8:
        for h in range(2):
            V = decode(b.v[b.table[0].long(), h]).reshape(-1, 128)[:L].abs().cumsum(0)[L - n:]
            tol[:, h * 5:h * 5 + 5] += (2.0 ** -32 - 2.0 ** -25) * V[:, None]
    out, lse = run(b, scale=scale)
    assert_close(out, want, tol, "out")
    assert_close(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("n,L", [(1, 60), (3, 2100), (100, 130), (150, 3000)])
def test_every_score_minus_infinity_gives_zeros_whatever_the_values(n, L):
    b = Batch([n], [L], 10, 2, 128, False, seed=n)
    b.k[:, :, :, 5] = -math.inf
    b.q[:, :, 5] = b.q[:, :, 5].abs() + 1
    for key, d, val in ((0, 3, math.inf), (17, 3, -math.inf), (40, 7, math.nan), (L - n, 9, math.inf)):
        p, r = place(b, 0, key)
        b.v[p, :, r, d] = val
    for max_q in (0, n):
        out, lse = run(b, max_q=max_q)
        assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,L", [(1, 200), (3, 5000), (100, 260), (100, 5000)])
def test_infinite_values_under_tiny_probabilities(D, n, L):
    # the key at `peak` is about 280 (natural) above the others: their probabilities are positive, but exp2 of the
    # distance is 0 in fp32, wherever the keys' maxima are joined
    for bad in (1, 33, 70, L // 2):
        b = Batch([n], [L], 8, 2, D, False, seed=n + D)
        peak = 5
        b.q[:, :, 0] = 16.0
        b.k[:, :, :, 0] = 0.0
        p, r = place(b, 0, peak)
        b.k[p, :, r, 0] = 280.0 / 16 * D ** 0.5
        p, r = place(b, 0, bad)
        b.v[p, :, r, 3], b.v[p, :, r, 7], b.v[p, :, r, D - 1] = math.inf, -math.inf, math.nan
        want, want_lse, tol, tol_lse = b.attention()
        for max_q in (0, n):
            out, lse = run(b, max_q=max_q)
            assert_close(out, want, tol, f"key {bad}, max_q {max_q}")
            assert_close(lse, want_lse, tol_lse)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("scale", [1e-30, 1e-37, 3e-39])
def test_smallest_softmax_scales(fp8, n, scale):
    b = Batch([n], [333], 8, 2, 128, fp8, seed=n)
    want, want_lse, tol, tol_lse = b.attention(scale)
    out, lse = run(b, scale=scale)
    assert_close(out, want, tol, "out")
    assert_close(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,L", [(1, 300), (1, 3000), (60, 300)])
@pytest.mark.parametrize("power", [20, 24, 28, 31, 36, 60])
def test_scores_of_every_size(fp8, sign, n, L, power):
    # scores are multiples of 2^power (exact products), so each row's answer is the value of its largest: any rounding
    # of scores of 16 * 2^power to fp32 stays below the 2^power between neighbours.  Nothing but that value
    # remains of the sum; it is rounded to bf16 once: 2^-8 of it.
    b = Batch([n], [L], 10, 2, 128, fp8, seed=power)
    level = torch.randint(1, 12, (L,), generator=b.g).float()
    level[7] = 15.0 if sign > 0 else 0.5
    one_channel_scores(b, sign * level)
    out, lse = run(b, scale=2.0 ** power)
    p, r = place(b, 0, 7)
    for h in range(2):
        want = decode(b.v[p, h, r])[None, None].expand(n, 5, 128)
        assert_close(out[:, h * 5:h * 5 + 5], want, 2.0 ** -8 * want.abs(), f"head {h}")
    top = sign * float(level[7]) * 2.0 ** power
    assert_close(lse, torch.full(lse.shape, top, dtype=torch.float64), torch.full(lse.shape, 2.0 ** -21 * abs(top), dtype=torch.float64))


@pytest.mark.parametrize("n,L", [(1, 700), (1, 5000), (100, 1000)])
def test_values_near_the_largest_bf16(n, L):
    # scores rise along the keys by less than the step at which old values are scaled down
    b = Batch([n], [L], 10, 2, 128, False, seed=n, v_gain=2.0 ** 121)
    one_channel_scores(b, torch.arange(L) / L * 5.25)
    want, _, tol, _ = b.attention(1.0)
    out, _ = run(b, scale=1.0)
    assert torch.isfinite(want).all()
    assert_close(out, want, tol)


@pytest.mark.parametrize("n,L", [(1, 100), (2, 5000), (100, 600), (300, 9000)])
@pytest.mark.parametrize("v_scale", [1e-39, 3e-37, 1e36])
def test_value_scales_of_every_size(n, L, v_scale):
    # values of 256 to 448; the bound is that of a scale of 1, in units of the scale (outputs and their tolerance
    # are normal numbers of bf16)
    b = Batch([n], [L], 10, 2, 128, True, seed=L)
    b.v = torch.randint(0x78, 0x7F, b.v.shape, generator=b.g, dtype=torch.uint8)
    b.vs = torch.ones(1)
    want, _, tol, _ = b.attention()
    b.vs = torch.full((1,), v_scale)
    want, tol = want * float(b.vs), tol * float(b.vs)
    out, _ = run(b)
    # 448e36 passes bf16's largest, 2^128 - 2^120, and what is half a step above that rounds to inf: a mean whose
    # whole tolerance lies there is inf, one whose tolerance reaches across may be
    edge = 2.0 ** 128 - 2.0 ** 119
    may = (want - tol < edge) & (want + tol >= edge)
    want = torch.where((want - tol >= edge) | (may & torch.isinf(out)), math.inf, want)
    assert_close(out, want, tol)

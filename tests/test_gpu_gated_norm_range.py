"""The gated norm of heads of every size and gates of every value, the same with and without a quantized output."""
import pytest
import torch

from tests.gdn_helpers import BF16, F32, HALF, assert_within, gated_norm, rand, uniform
from tests.gpu_helpers import DEV, nv

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def both(x, z, w, eps, **kw):
    """The rows without a quantized output and beside one."""
    x, z, w = (t.to(DEV) for t in (x, z, w))
    return nv().gated_rms_norm(x, z, w, eps=eps, out_dtype=F32)[0], nv().gated_rms_norm(x, z, w, eps=eps, out_dtype=F32, quant="fp8", **kw)


@pytest.mark.parametrize("T,H,D", [(3, 2, 16), (5, 3, 128), (4, 1, 1024), (3, 40, 128)])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("size", [1e12, 1e15, 1e18, 1.6e18, 1e20, 1e30, 5e37])
@pytest.mark.parametrize("gate", [3.0, 1e6])
def test_large_heads(T, H, D, xt, size, gate):
    x, z, w = rand(T, H, D, seed=51, dtype=F32), rand(T, H, D, seed=52, scale=gate), 0.5 + uniform(D, seed=53)
    x[1] *= size                                # beside heads of order 1
    x = x.to(xt)
    want, tol32, tol = (t.flatten(1) for t in gated_norm(x, z, w, 1e-6))
    plain, (y, _) = both(x, z, w, 1e-6)
    assert_within(plain, want, tol32 + HALF[F32] * want.abs(), "plain")
    assert_within(y, want, tol + HALF[F32] * want.abs(), "quantized")


@pytest.mark.parametrize("T,H,D", [(3, 2, 16), (5, 3, 128), (4, 1, 1024)])
@pytest.mark.parametrize("size", [1e-12, 1e-18, 1e-22, 1e-30, 1e-36])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_small_heads(T, H, D, size, eps):
    x, z, w = rand(T, H, D, seed=54, dtype=F32), rand(T, H, D, seed=55, scale=2.0), 0.5 + uniform(D, seed=56)
    x[1] *= size
    want, tol32, tol = (t.flatten(1) for t in gated_norm(x, z, w, eps))
    plain, (y, _) = both(x, z, w, eps)
    assert_within(plain, want, tol32 + HALF[F32] * want.abs(), "plain")
    assert_within(y, want, tol + HALF[F32] * want.abs(), "quantized")


def test_heads_of_zeros():
    x, z, w = rand(4, 3, 64, seed=57), rand(4, 3, 64, seed=58), torch.ones(64)
    x[1, 1], x[2] = 0.0, 0.0
    for eps in (1e-6, 1e-30):
        plain, (y, _) = both(x, z, w, eps)
        assert (plain[1, 64:128] == 0).all() and (plain[2] == 0).all() and torch.isfinite(plain).all()
        assert (y[1, 64:128] == 0).all() and (y[2] == 0).all() and torch.isfinite(y).all()
    plain, (y, _) = both(x, z, w, 0.0)          # 0 / 0
    assert torch.isnan(plain[2]).all() and torch.isnan(y[2]).all() and torch.isfinite(plain[0]).all() and torch.isfinite(y[0]).all()


@pytest.mark.parametrize("zt", [BF16, F32])
def test_gates_that_are_not_finite(zt):
    # z sigmoid(z): infinity at infinity; at minus infinity -inf * 0, which is not a number
    x, w = torch.ones(1, 2, 64), torch.ones(64)
    z = rand(1, 2, 64, seed=59, dtype=F32).to(zt)
    z[0, 0, 3], z[0, 0, 20], z[0, 1, 40] = -INF, INF, NAN
    want = gated_norm(x, z, w, 1e-6)[0].flatten(1)
    assert torch.isnan(want[0, 3]) and want[0, 20] == INF and torch.isnan(want[0, 104])
    plain, (y, q) = both(x, z, w, 1e-6, mode="given", scale=torch.full((1,), 0.02, device=DEV))
    for got in (plain, y):
        assert_within(got, want, 2.0 ** -18 * want.abs())
    codes = q.codes.cpu()[0]
    assert (codes[[3, 104]] & 0x7F).tolist() == [0x7F, 0x7F] and codes[20] == 0x7E
    s = torch.full((1,), 0.02, device=DEV)
    y, q = nv().gated_rms_norm(x.to(DEV), z.to(DEV), w.to(DEV), out_dtype=F32, quant="nvfp4", mode="given", scale=s)
    assert_within(y, want, 2.0 ** -18 * want.abs())
    alone = nv().quantize(y, "given", s)        # the quantizer's bytes, whatever it makes of them
    assert torch.equal(q.codes, alone.codes) and torch.equal(q.scales, alone.scales)

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

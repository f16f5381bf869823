"""Head norms and rotation in fp32 are no less exact than the plain form in fp32, root mean square over many vectors."""
import pytest
import torch

from tests.gpu_helpers import DEV, nv
from tests.paged_helpers import norm_rope, rope_table

pytestmark = pytest.mark.gpu


def plain(x, w, row, interleaved, eps=1e-6):
    """The formula step by step in fp32."""
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    R = row.shape[-1]
    c, n = row[:, None, :R // 2], row[:, None, R // 2:]
    ia, ib = (torch.arange(0, R, 2), torch.arange(1, R, 2)) if interleaved else (torch.arange(R // 2), torch.arange(R // 2, R))
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * n, b * c + a * n
    return y


@pytest.mark.parametrize("D,R,interleaved", [(64, 64, False), (128, 128, False), (256, 64, True)])
@pytest.mark.parametrize("gain", [1e-2, 1.5, 300.0])
def test_error_is_not_above_the_plain_forms(D, R, interleaved, gain):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(1500, 4, D, generator=g) * gain
    w = 1 + 0.2 * torch.randn(D, generator=g)
    table, pos = rope_table(400, R), torch.randint(0, 400, (1500,), generator=g, dtype=torch.int32)
    want, _ = norm_rope(x, w, table, pos, interleaved)
    got, _ = nv().qk_norm_rope(x.to(DEV), q_weight=w.to(DEV), rope=table.to(DEV), positions=pos.to(DEV), interleaved=interleaved)
    err = lambda y: ((y.double() - want).norm() / want.norm()).item()  # noqa: E731
    form = plain(*(t.to(DEV) for t in (x, w, table[pos.long()])), interleaved)
    assert err(got.cpu()) <= err(form.cpu())


def test_vectors_whose_mean_square_is_no_ordinary_number():
    # zeros, subnormal means and ones past fp32's range, without and with eps; x / sqrt(mean + eps) w in 64 bits where
    # the fp32 sum of squares is finite and normal, else as fp32 gives it: 0 / 0 and inf are NaN and 0
    D = 128
    x = torch.zeros(7, 1, D)
    x[1], x[2], x[3], x[4] = 1e-18, 2e-16, 1e15, 1e18
    x[5] = 1e25                              # its mean square is inf: outputs 0
    x[6, :, 3] = float("inf")
    w = torch.ones(D)
    for eps in (0.0, 1e-6):
        got = nv().qk_norm_rope(x.to(DEV), q_weight=w.to(DEV), eps=eps)[0].cpu().double()
        want, tol = norm_rope(x, w, None, None, False, eps)
        for t in (1, 2, 3, 4):
            assert ((got[t] - want[t]).abs() <= tol[t] + 1e-38).all(), (eps, t)
        assert torch.isnan(got[0]).all() if eps == 0 else (got[0] == 0).all()
        assert (got[5] == 0).all()
        assert torch.isnan(got[6, 0, 3]) and (got[6, 0, torch.arange(D) != 3] == 0).all()

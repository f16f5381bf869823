"""Norms with quantized outputs against the 64-bit formula and the quantizer's oracle: types, widths from one block to
the largest, strides, in-place residuals, rows of zeros, infinities and NaN."""
import pytest
import torch

from oracle import nvfp4_ref as ref
from tests.gdn_helpers import BF16, F32, HALF, add_norm, add_norm64, assert_within, check_quant, gated_norm, rand, uniform
from tests.gpu_helpers import DEV, assert_quant_equal, nv

pytestmark = pytest.mark.gpu


def gpu(x):
    return None if x is None else x.to(DEV)


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (1, 5120), (5, 1040), (2, 16384), (2, 16400), (1, 32768), (300, 256)])
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16), (BF16, None), (F32, None)])
def test_add_rms_norm(rows, cols, xt, rt):
    x = rand(rows, cols, seed=1, dtype=xt, scale=1.5)
    r = None if rt is None else rand(rows, cols, seed=2, dtype=rt, scale=3.0)
    w = 0.5 + uniform(cols, seed=3)
    r_want, y64 = add_norm64(x, r, w, 1e-6)
    y32 = y64.float()
    for quant, mode in (("nvfp4", "per_row"), ("nvfp4", "given"), ("fp8", "per_row"), ("fp8", "given")):
        given = 0.013
        s = torch.full((1,), given, device=DEV) if mode == "given" else None
        y, q, r_out = nv().add_rms_norm(gpu(x), gpu(w), gpu(r), out_dtype=F32, quant=quant, mode=mode, scale=s)
        assert_within(y, y32.double(), U_ONE * y32.double().abs())
        assert (r_out is None) if r is None else torch.equal(r_out.cpu(), r_want)
        if quant == "nvfp4":
            check_quant(q, y.cpu(), quant, mode, given)          # of the same launch's fp32 output
        check_quant(q, y64, quant, mode, given)                  # and of the formula's
        alone = nv().add_rms_norm(gpu(x), gpu(w), gpu(r), out_dtype=None, quant=quant, mode=mode, scale=s)
        assert alone[0] is None and torch.equal(alone[1].codes, q.codes)
    yb, none, _ = nv().add_rms_norm(gpu(x), gpu(w), gpu(r))
    assert none is None and torch.equal(yb.cpu(), y32.to(BF16))


U_ONE = 2.0 ** -24 * 1e-3    # fl32 of the formula: equal but where 64 bits themselves land on a border


def test_in_place_strided_and_given_outputs():
    rows, cols = 37, 512
    fused = gpu(rand(rows, 3 * cols, seed=4))
    x, res = fused[:, cols:2 * cols], gpu(rand(rows, cols + 64, seed=5, scale=2.0))[:, :cols]
    w = gpu(0.5 + uniform(cols, seed=3))
    r_want, y32 = add_norm(x.cpu(), res.cpu(), w.cpu(), 1e-5)
    before = fused.clone()
    out = torch.full((rows, cols + 32), 7.0, dtype=BF16, device=DEV)
    y, q, r = nv().add_rms_norm(x, w, res, eps=1e-5, out=out[:, :cols], quant="nvfp4", residual_out=res)
    assert y.data_ptr() == out.data_ptr() and r is res
    assert torch.equal(res.cpu(), r_want) and torch.equal(y.cpu(), y32.to(BF16)) and (out[:, cols:] == 7.0).all()
    assert torch.equal(fused, before)
    again = nv().NVFP4Tensor(torch.empty_like(q.codes), torch.empty_like(q.scales), torch.empty_like(q.global_scale))
    got = nv().add_rms_norm(res, w, eps=1e-5, out_dtype=None, quant="nvfp4", q_out=again)[1]
    assert got is again
    assert_quant_equal(got, ref.quantize(add_norm(res.cpu(), None, w.cpu(), 1e-5)[1].numpy(), ref.PER_ROW))
    # the norm over its own input
    want = nv().add_rms_norm(x.contiguous(), w, eps=1e-5)[0]
    nv().add_rms_norm(x, w, eps=1e-5, out=x)
    assert torch.equal(x, want)


def some_rows(q, quant, rows):
    if quant == "nvfp4":
        return nv().NVFP4Tensor(q.codes[rows], q.scales[rows], q.global_scale[rows])
    return nv().FP8Tensor(q.codes[rows], q.scale[rows])


@pytest.mark.parametrize("quant", ["nvfp4", "fp8"])
def test_rows_of_zeros_and_tiny_rows(quant):
    x = torch.zeros(4, 64)
    x[1, 3], x[2], x[3, 0] = -0.0, 1e-30, -3e38
    w = torch.ones(64)
    y, q, _ = nv().add_rms_norm(gpu(x), gpu(w), eps=1e-6, out_dtype=F32, quant=quant)
    assert (y[:2] == 0).all() and torch.isfinite(y).all()
    check_quant(some_rows(q, quant, slice(2, 4)), add_norm64(x[2:], None, w, 1e-6)[1], quant, "per_row", None)
    if quant == "nvfp4":
        assert_quant_equal(q, ref.quantize(y.cpu().numpy(), ref.PER_ROW))
        assert (q.scales[:2] == 0).all() and (q.codes[0] == 0).all() and q.global_scale[0] == 0
    if quant == "fp8":
        assert q.scale[0] == 0 and (q.codes[0] == 0).all() and q.codes[1, 3] == 0x80


@pytest.mark.parametrize("quant", ["nvfp4", "fp8"])
def test_non_finite_rows_are_reported_and_stay_alone(quant):
    x = rand(5, 128, seed=6, dtype=F32)
    x[1, 5], x[3, 7] = float("nan"), float("inf")
    w = 0.5 + uniform(128, seed=3)
    y, q, _ = nv().add_rms_norm(gpu(x), gpu(w), out_dtype=F32, quant=quant)
    s = (q.global_scale if quant == "nvfp4" else q.scale).cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(s[1]) and not torch.isfinite(s[3])
    ok = [0, 2, 4]
    _, y32 = add_norm(x[ok], None, w, 1e-6)
    assert torch.equal(y[ok].cpu(), y32) and torch.isfinite(s[ok]).all()
    if quant == "nvfp4":
        assert_quant_equal(nv().NVFP4Tensor(q.codes[ok], q.scales[ok], q.global_scale[ok]), ref.quantize(y32.numpy(), ref.PER_ROW))


@pytest.mark.parametrize("T,H,D", [(1, 1, 16), (1, 32, 128), (7, 5, 64), (3, 2, 1024), (130, 48, 128), (2, 256, 128), (9, 3, 32)])
@pytest.mark.parametrize("xt,zt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_gated_rms_norm(T, H, D, xt, zt):
    x, w = rand(T, H, D, seed=7, dtype=xt, scale=0.3), 0.5 + uniform(D, seed=8)
    fused = rand(T, 3 * H * D, seed=9, dtype=zt, scale=3.0)
    z = fused[:, H * D:2 * H * D].unflatten(1, (H, D))
    zg = gpu(fused)[:, H * D:2 * H * D].unflatten(1, (H, D))
    want, tol32, tol = (t.flatten(1) for t in gated_norm(x, z, w, 1e-6))
    y, q, = nv().gated_rms_norm(gpu(x), zg, gpu(w), out_dtype=F32, quant="nvfp4")
    assert_within(y, want, tol + HALF[F32] * want.abs())
    check_quant(q, y.cpu(), "nvfp4", "per_row", None)
    for quant, mode in (("nvfp4", "given"), ("fp8", "per_row"), ("fp8", "given")):
        s = torch.full((1,), 0.02, device=DEV) if mode == "given" else None
        none, q = nv().gated_rms_norm(gpu(x), zg, gpu(w), out_dtype=None, quant=quant, mode=mode, scale=s)
        assert none is None
        check_quant(q, want, quant, mode, 0.02)
    for dtype in (BF16, F32):
        y, none = nv().gated_rms_norm(gpu(x), zg, gpu(w), out_dtype=dtype)
        assert none is None
        assert_within(y, want, tol32 + HALF[dtype] * want.abs())


def test_gate_of_every_size():
    z = torch.tensor([0.0, -0.0, 1e-30, 88.0, 89.0, -87.0, -88.0, -89.0, -200.0, 200.0, 3e38, -3e38, 20.0, -20.0, 1.0, -1.0])
    x = torch.ones(1, 1, 16)
    want, *tols = (t.flatten(1) for t in gated_norm(x, z[None, None], torch.ones(16), 1e-6))
    for quant, tol in zip(("none", "fp8"), tols):
        y, _ = nv().gated_rms_norm(gpu(x), gpu(z)[None, None], torch.ones(16, device=DEV), out_dtype=F32, quant=quant)
        assert_within(y, want, tol + HALF[F32] * want.abs())


def test_no_rows():
    w = torch.ones(64, device=DEV)
    y, q, r = nv().add_rms_norm(torch.empty(0, 64, device=DEV), w, torch.empty(0, 64, device=DEV), quant="nvfp4")
    assert y.shape == (0, 64) and q.codes.shape == (0, 32) and r.shape == (0, 64)
    y, q = nv().gated_rms_norm(torch.empty(0, 2, 64, device=DEV), torch.empty(0, 2, 64, device=DEV), w, quant="fp8")
    assert y.shape == (0, 128) and q.codes.shape == (0, 128)


@pytest.mark.parametrize("rows", [1, 3, 67, 1000])
@pytest.mark.parametrize("cols", [16, 32, 80, 256, 528, 1008, 1024])
@pytest.mark.parametrize("eps", [0.0, 1e-3])
def test_short_rows_share_wavefronts(rows, cols, eps):
    x, w = rand(rows, cols, seed=10, scale=2.0), 0.5 + uniform(cols, seed=11)
    _, y64 = add_norm64(x, None, w, eps)
    y32 = y64.float()
    for quant in ("nvfp4", "fp8"):
        y, q, _ = nv().add_rms_norm(gpu(x), gpu(w), eps=eps, out_dtype=F32, quant=quant)
        assert torch.equal(y.cpu(), y32)
        check_quant(q, y64, quant, "per_row", None)
    assert torch.equal(nv().add_rms_norm(gpu(x), gpu(w), eps=eps)[0].cpu(), y32.to(BF16))


@pytest.mark.parametrize("T,H,D", [(1, 3, 16), (67, 5, 16), (1000, 2, 64), (300, 3, 64), (129, 7, 128), (33, 64, 16), (5, 65, 16), (3, 9, 128)])
@pytest.mark.parametrize("eps", [0.0, 1e-3])
def test_short_rows_of_heads(T, H, D, eps):
    x, z, w = rand(T, H, D, seed=12), rand(T, H, D, seed=13, scale=2.0), 0.5 + uniform(D, seed=14)
    want, tol32, tol = (t.flatten(1) for t in gated_norm(x, z, w, eps))
    for quant in ("nvfp4", "fp8"):
        y, q = nv().gated_rms_norm(gpu(x), gpu(z), gpu(w), eps=eps, out_dtype=F32, quant=quant)
        assert_within(y, want, tol + HALF[F32] * want.abs())
        check_quant(q, want, quant, "per_row", None)
    assert_within(nv().gated_rms_norm(gpu(x), gpu(z), gpu(w), eps=eps)[0], want, tol32 + HALF[BF16] * want.abs())


@pytest.mark.parametrize("given", [None, 2.0 ** -6, 0.013])
def test_fp8_bytes_next_to_borders(given):
    # quotients that lie on a border between two E4M3 values, or a rounding in fp32 away from it
    x = torch.full((64, 256), 0.5, dtype=F32)
    steps = torch.arange(256, dtype=torch.float64)
    border = (1 + (2 * (steps % 8) + 1) / 16) * 2.0 ** (steps // 8 % 12 - 6)
    w = (border * (1 + 2.0 ** -23 * (steps // 96 - 1))).float()
    x[:, 0] = 1.0 + torch.arange(64) * 2.0 ** -18              # norms that differ in their last bits
    _, y64 = add_norm64(x, None, w, 0.0)
    s = None if given is None else torch.full((1,), given, device=DEV)
    _, q, _ = nv().add_rms_norm(gpu(x), gpu(w), eps=0.0, out_dtype=None, quant="fp8", mode="per_row" if given is None else "given", scale=s)
    check_quant(q, y64, "fp8", "per_row" if given is None else "given", given)
    z = gpu(torch.full((64, 4, 64), 1.5))
    _, q = nv().gated_rms_norm(gpu(x).unflatten(1, (4, 64)), z, gpu(w[:64]), eps=0.0, out_dtype=None, quant="fp8",
                               mode="per_row" if given is None else "given", scale=s)
    want = gated_norm(x.unflatten(1, (4, 64)), z.cpu(), w[:64], 0.0)[0].flatten(1)
    check_quant(q, want, "fp8", "per_row" if given is None else "given", given)

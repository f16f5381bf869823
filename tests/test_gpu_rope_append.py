"""Per-head norms with the position rotation, and appending to the paged cache, against the plain 64-bit
implementation: types, head layouts, head sizes, partial and interleaved rotation, strides, ragged and
padded batches, places without a page."""
import numpy as np
import pytest
import torch

from oracle import nvfp4_ref as ref
from tests.gpu_helpers import DEV, nv
from tests.paged_helpers import Batch, E4M3, assert_close, decode, norm_rope, rope_table, stored

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed=0, dtype=BF16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * 1.7).to(dtype)


def gpu(x):
    return None if x is None else x.to(DEV)


@pytest.mark.parametrize("D,R", [(16, 16), (64, 32), (80, 48), (128, 128), (128, 96), (256, 64), (512, 512)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("xt,ot", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_norm_rope(D, R, interleaved, xt, ot):
    T, Hq, Hk = 7, 5, 2
    q, k = rand(T, Hq, D, seed=1, dtype=xt), rand(T, Hk, D, seed=2, dtype=xt)
    qw, kw = 1 + 0.3 * rand(D, seed=3, dtype=F32), 1 + 0.3 * rand(D, seed=4, dtype=F32)
    table = rope_table(300, R)
    pos = torch.tensor([0, 1, 299, 17, 17, 256, 100], dtype=torch.int32)
    gq, gk = nv().qk_norm_rope(gpu(q), gpu(k), gpu(qw), gpu(kw), gpu(table), gpu(pos), interleaved=interleaved, out_dtype=ot)
    for got, x, w in ((gq, q, qw), (gk, k, kw)):
        y, tol = norm_rope(x, w, table, pos, interleaved)
        assert got.dtype == ot
        assert_close(got, y, stored(y, tol, ot))


@pytest.mark.parametrize("T,Hq,Hk", [(1, 40, 8), (1, 1, 1), (333, 7, 3), (2, 128, 1)])
@pytest.mark.parametrize("weights,rope", [(True, False), (False, True), (False, False)])
def test_parts_left_out(T, Hq, Hk, weights, rope):
    D = 128
    q, k = rand(T, Hq, D, seed=5), rand(T, Hk, D, seed=6)
    w = 1 + 0.3 * rand(D, seed=3, dtype=F32) if weights else None
    table = rope_table(64, D) if rope else None
    pos = (torch.arange(T) % 64).to(torch.int32) if rope else None
    gq, gk = nv().qk_norm_rope(gpu(q), gpu(k), gpu(w), None, gpu(table), gpu(pos))
    for got, x, wt in ((gq, q, w), (gk, k, None)):
        y, tol = norm_rope(x, wt, table, pos, False)
        assert_close(got, y, stored(y, tol, BF16))
    alone, none = nv().qk_norm_rope(gpu(q), None, gpu(w), None, gpu(table), gpu(pos))
    assert none is None and torch.equal(alone, gq)


def test_strided_views_in_place_and_untouched_neighbours():
    T, Hq, Hk, D = 50, 6, 2, 128
    fused = rand(T, (Hq + 2 * Hk) * D, seed=7)
    w, table, pos = 1 + 0.3 * rand(D, seed=3, dtype=F32), rope_table(64, D), torch.arange(T, dtype=torch.int32)
    f = gpu(fused)
    q, k = f[:, :Hq * D].unflatten(1, (Hq, D)), f[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    want = nv().qk_norm_rope(q.contiguous(), k.contiguous(), gpu(w), gpu(w), gpu(table), gpu(pos))
    heads_first = torch.empty((Hq, T, D), dtype=BF16, device=DEV).transpose(0, 1)
    got = nv().qk_norm_rope(q, k, gpu(w), gpu(w), gpu(table), gpu(pos), q_out=heads_first)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    nv().qk_norm_rope(q, k, gpu(w), gpu(w), gpu(table), gpu(pos), q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(f[:, (Hq + Hk) * D:].cpu(), fused[:, (Hq + Hk) * D:])


def test_positions_outside_the_table_become_nan():
    D, R = 128, 64
    q, table = rand(4, 3, D, seed=8), rope_table(10, R)
    pos = torch.tensor([9, 10, -1, 2 ** 31 - 1], dtype=torch.int32)
    for inter in (False, True):
        got, _ = nv().qk_norm_rope(gpu(q), rope=gpu(table), positions=gpu(pos), interleaved=inter)
        y, tol = norm_rope(q, None, table, pos, inter)
        assert_close(got, y, stored(y, tol, BF16))
        assert torch.isnan(got[1:, :, :R]).all() and torch.equal(got[1:, :, R:].cpu(), q[1:, :, R:])


def test_zero_and_huge_vectors():
    D = 128
    q = torch.zeros(3, 2, D, dtype=F32)
    q[1] = 1e18
    q[2, :, ::2] = 1e-20
    w = torch.ones(D)
    got, _ = nv().qk_norm_rope(gpu(q), q_weight=gpu(w), eps=1e-6)
    y, tol = norm_rope(q, w, None, None, False)
    assert_close(got, y, stored(y, tol, F32))
    assert nv().qk_norm_rope(gpu(q[:0]))[0].shape == (0, 2, D)


def append_case(b, xt=BF16, R=None, weights=True, with_q=True, interleaved=False, positions=None, q_out_dtype=BF16):
    """Appends random keys and values to the batch's cache and checks every byte of it."""
    D, Hk, Hq, T = b.D, b.Hk, b.Hq, b.T
    kv, kv_len, cu, _ = b.device()
    before = kv.k.clone(), kv.v.clone()
    # keys and values are column ranges of one projection
    f = rand(T, (Hq + 2 * Hk) * D, seed=21, dtype=xt)
    q, k, v = (x.unflatten(1, (-1, D)) for x in (f[:, :Hq * D], f[:, Hq * D:(Hq + Hk) * D], f[:, (Hq + Hk) * D:]))
    g = gpu(f)
    gq, gk, gv = (x.unflatten(1, (-1, D)) for x in (g[:, :Hq * D], g[:, Hq * D:(Hq + Hk) * D], g[:, (Hq + Hk) * D:]))
    kw = 1 + 0.3 * rand(D, seed=3, dtype=F32) if weights else None
    qw = 1 + 0.3 * rand(D, seed=4, dtype=F32) if weights and with_q else None
    table = rope_table(4096, R) if R else None
    q_out = torch.full((T, Hq, D), 5.0, dtype=q_out_dtype, device=DEV) if with_q else None
    nv().kv_append(kv, gk, gv, kv_len, cu, k_weight=gpu(kw), rope=gpu(table), positions=gpu(positions), interleaved=interleaved,
                   q=gq if with_q else None, q_weight=gpu(qw), q_out=q_out)
    torch.cuda.synchronize()
    place = torch.full((T,), -(10 ** 9), dtype=torch.int64)
    seq = torch.full((T,), -1, dtype=torch.int64)
    for s, n in enumerate(b.new):
        c0 = int(b.cu[s])
        place[c0:c0 + n] = b.kv[s] - n + torch.arange(n)
        seq[c0:c0 + n] = s
    pos = place if positions is None else positions.long()
    yk, tk = norm_rope(k, kw, table, pos, interleaved)
    if with_q:
        yq, tq = norm_rope(q, qw, table, pos, interleaved)
        mine = seq >= 0
        assert_close(q_out.cpu()[mine], yq[mine], stored(yq, tq, q_out_dtype)[mine], "q")
        assert (q_out.cpu()[~mine] == 5.0).all()
    want_k, want_v = before[0].cpu().clone(), before[1].cpu().clone()
    got_k, got_v = kv.k.cpu(), kv.v.cpu()
    for t in range(T):
        if seq[t] < 0 or place[t] < 0 or place[t] // b.page >= b.width:
            continue
        p, r = int(b.table[seq[t], place[t] // b.page]), int(place[t]) % b.page
        if not 0 <= p < want_k.shape[0]:
            continue
        if b.fp8:
            for h in range(Hk):
                ks, vs = b.scales(h)
                y, e = yk[t, h] / ks, tk[t, h] / ks + 4 * 2.0 ** -24 * yk[t, h].abs() / ks
                half = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64))
                x = decode(got_k[p, h, r])
                sat = y.abs() >= 448
                ok = torch.where(torch.isnan(y), torch.isnan(x), torch.where(sat, x.abs() >= 448 * (1 - 2 ** -4), (x - y).abs() <= half + e))
                assert ok.all(), (t, h, x[~ok][:3], y[~ok][:3])
                want_k[p, h, r] = got_k[p, h, r]
                want_v[p, h, r] = torch.from_numpy(ref.fp8_kv_quantize(v[t, h].float().numpy(), np.float32(vs)))
        else:
            assert_close(got_k[p, :, r], yk[t], stored(yk[t], tk[t], BF16), f"k of token {t}")
            want_k[p, :, r] = got_k[p, :, r]
            want_v[p, :, r] = v[t].to(BF16)
    bits = lambda x: x if x.dtype == torch.uint8 else x.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(got_v), bits(want_v)), "values, or bytes outside the appended places"
    assert torch.equal(bits(got_k), bits(want_k)), "bytes of k outside the appended places"


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (64, 32, True), (256, 64, False), (80, 16, True)])
def test_append(fp8, xt, D, R, inter):
    append_case(Batch([5, 1, 0, 40, 1], [5, 33, 7, 90, 1], 6, 2, D, fp8, seed=D), xt, R, interleaved=inter)


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("joint", [True, False])
def test_append_pages_and_one_allocation(page, joint):
    append_case(Batch([70, 3], [page + 40, page * 2], 4, 2, 128, True, page=page, joint=joint, per_head=True, seed=2), R=128)


def test_append_without_queries_norm_or_rotation():
    b = Batch([1] * 70, [1 + 3 * i for i in range(70)], 8, 4, 128, True, seed=3)
    append_case(b, with_q=False)
    append_case(b, with_q=False, weights=False)
    append_case(b, weights=False, R=128, q_out_dtype=F32)


def test_append_given_positions():
    b = Batch([4, 2], [10, 6], 4, 2, 128, True, seed=4)
    append_case(b, R=64, positions=torch.tensor([0, 4095, 7, 7, 4096, -3], dtype=torch.int32))


def test_append_rows_of_nobody_and_places_without_a_page():
    b = Batch([6, 5, 3], [4, 200, 30], 4, 2, 128, True, lead=3, tail=4, seed=5)     # two tokens before place 0
    b.table[1, 199 // 16] = -1
    b.table[2, 1] = b.k.shape[0]
    append_case(b, R=128)
    b = Batch([6, 5], [20, 40], 4, 2, 128, False, seed=6)
    b.kv_len[1], b.kv[1] = 51, 51                                                     # past the table's three pages
    append_case(b, R=128)


def test_append_many_sequences():
    append_case(Batch([1] * 300, [1 + i % 40 for i in range(300)], 2, 1, 64, True, seed=7), R=64)


def test_append_single_token_single_head():
    append_case(Batch([1], [1], 1, 1, 128, True, seed=8), R=128)


def test_append_values_round_as_the_codec():
    # every bf16 value as v, bit for bit the codec's bytes
    D = 128
    x = (torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)).view(BF16).reshape(512, 1, D)
    b = Batch([512], [512], 1, 1, D, True, seed=9)
    kv, kv_len, cu, _ = b.device()
    nv().kv_append(kv, gpu(x), gpu(x), kv_len, cu)
    codec_k, codec_v = (nv().fp8_kv_quantize(gpu(x), s) for s in (kv.k_scale, kv.v_scale))
    rows = kv.page_table[0].long()
    assert torch.equal(kv.v[rows].reshape(512, 1, D), codec_v)
    assert torch.equal(kv.k[rows].reshape(512, 1, D), codec_k)


def test_lengths_on_the_device_beyond_the_operands():
    b = Batch([3, 2], [40, 33], 8, 2, 128, True, seed=11)
    kv, _, _, q = b.device()
    k = torch.randn(5, 2, 128, device=DEV).to(BF16)
    for kv_len, cu in (([10 ** 9, -5], [0, 3, 5]), ([40, 33], [0, 10 ** 9, 5]), ([40, 33], [-4, 3, 2]), ([2 ** 31 - 1] * 2, [5, 0, 5]),
                       ([-2 ** 31] * 2, [0, 2 ** 31 - 1, 5])):
        nv().kv_append(kv, k, k, torch.tensor(kv_len, dtype=torch.int32, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV),
                       rope=gpu(rope_table(8, 128)))
        torch.cuda.synchronize()

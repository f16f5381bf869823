"""The paged cache's operators on batches whose kernels small ones do not reach: appends and norms of so many tokens that a
wavefront takes two groups of heads, tiles of very uneven lengths, lengths on the device that are out of range
beside memory that must not change, and the layer's output through the quantized output projection by value."""
import pytest
import torch

from oracle import nvfp4_ref as ref
from tests.gpu_helpers import DEV, assert_gemm_close, assert_quant_equal, nv, to_host
from tests.paged_helpers import Batch, assert_close, norm_rope, rope_table, stored
from tests.test_gpu_paged_attention import check
from tests.test_gpu_paged_steps import BF16, Layer
from tests.test_gpu_rope_append import F32, append_case, gpu, rand

pytestmark = pytest.mark.gpu


# ---- two groups of heads a wavefront: bf16 inputs from 16384 groups in all ---------------------------------------
# (a group is 512 / D heads of one kind, D taken up to a power of two; rounded up for each kind)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D,Hq,Hk,R,inter,T", [
    (256, 1, 4, 256, False, 3301),       # groups q, k k, v v: wavefronts over q|k, k|v and a last one alone
    (128, 9, 5, 32, True, 2399),         # q q q, k k, v v, the last of each kind not full
    (512, 3, 2, 512, False, 2401),       # one head a group
    (80, 2, 1, 48, False, 5501),         # lanes past the head's end
])
def test_long_append(fp8, D, Hq, Hk, R, inter, T):
    # several sequences, rows of nobody, places without a page and before the first, per-head scales
    b = Batch([T - 700, 0, 600, 93], [T - 703, 5, 640, 200], Hq, Hk, D, fp8, page=32, lead=2, tail=5, per_head=True, seed=T)
    b.table[2, 3] = -1
    b.table[3, 5] = b.k.shape[0]
    per = 512 // (1 << (D - 1).bit_length())
    assert b.T * (-(-Hq // per) + 2 * -(-Hk // per)) >= 16384
    append_case(b, R=R, interleaved=inter)


def test_long_append_without_queries_one_scale_given_positions():
    T = 8300                             # groups k, v: the scale and the weight change inside each wavefront
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-1, 4097, (T,), generator=g, dtype=torch.int32)
    append_case(Batch([T], [T + 9], 4, 1, 64, True, page=64, seed=1), with_q=False, R=64, positions=pos)


@pytest.mark.parametrize("D,Hq,Hk,R,inter", [(128, 9, 2, 128, False), (256, 5, 3, 64, True)])
def test_long_norm_rope(D, Hq, Hk, R, inter):
    T = 5501
    q, k = rand(T, Hq, D, seed=1), rand(T, Hk, D, seed=2)
    qw, kw = 1 + 0.3 * rand(D, seed=3, dtype=F32), 1 + 0.3 * rand(D, seed=4, dtype=F32)
    table, pos = rope_table(300, R), (torch.arange(T) * 7 % 301).to(torch.int32)          # 300 has no row: NaN
    for ot in (BF16, F32):
        got = nv().qk_norm_rope(gpu(q), gpu(k), gpu(qw), gpu(kw), gpu(table), gpu(pos), interleaved=inter, out_dtype=ot)
        for y, x, w in ((got[0], q, qw), (got[1], k, kw)):
            want, tol = norm_rope(x, w, table, pos, inter)
            assert_close(y, want, stored(want, tol, ot))
    one = nv().qk_norm_rope(gpu(q[:40]), gpu(k[:40]), gpu(qw), gpu(kw), gpu(table), gpu(pos[:40]), interleaved=inter)
    many = nv().qk_norm_rope(gpu(q), gpu(k), gpu(qw), gpu(kw), gpu(table), gpu(pos), interleaved=inter)
    bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(one[0]), bits(many[0][:40])) and torch.equal(bits(one[1]), bits(many[1][:40]))


# ---- tiles of uneven lengths --------------------------------------------------------------------------------------


@pytest.mark.parametrize("D,fp8", [(64, True), (128, True), (128, False), (256, False)])
@pytest.mark.parametrize("window", [0, 300])
def test_one_long_chunk_among_short_ones(D, fp8, window):
    # the longest tile has many times the mean's blocks; empty sequences and single tokens between
    new, kv = [90, 1, 0, 61, 33, 1, 200], [6100, 2500, 40, 61, 40, 3, 230]
    for max_q in (0, 200):
        check(Batch(new, kv, 8, 2, D, fp8, seed=D, tail=1), window=window, max_q=max_q)


# ---- lengths out of range ------------------------------------------------------------------------------------------


def guarded(x: torch.Tensor, n: int, fill):
    """x in the middle of a buffer with n more entries of the first dimension on either side: (view, whole buffer)."""
    big = torch.full((x.shape[0] + 2 * n, *x.shape[1:]), fill, dtype=x.dtype, device=DEV)
    big[n:n + x.shape[0]] = x.to(DEV)
    return big[n:n + x.shape[0]], big


def edges_kept(big: torch.Tensor, n: int, fill) -> bool:
    return bool((big[:n] == fill).all() and (big[-n:] == fill).all())


@pytest.mark.parametrize("Hq", [8, 2])
@pytest.mark.parametrize("kv_len,cu,new,kv", [
    ([10 ** 9, -5], [0, 3, 5], [3, 2], [48, 0]),              # the table's capacity; an empty cache
    ([2 ** 31 - 1, -2 ** 31], [0, 3, 5], [3, 2], [48, 0]),
    ([40, 33], [0, 10 ** 9, 5], [5, 0], [40, 33]),            # the last row; then a decreasing offset: no rows
    ([40, 33], [0, 2 ** 31 - 1, 2 ** 31 - 1], [5, 0], [40, 33]),
    ([40, 33], [-4, 3, 2], [3, 0], [40, 33]),
    ([40, 33], [-2 ** 31, 3, 5], [3, 2], [40, 33]),
])
def test_attention_of_lengths_out_of_range(Hq, kv_len, cu, new, kv):
    b = Batch(new, [48, 48], Hq, 2, 128, True, seed=11, tail=5 - sum(new))
    dev, _, _, q = b.device()
    k, kbig = guarded(b.k, 2, 0x7F)                            # NaN around the pool
    v, vbig = guarded(b.v, 2, 0x7F)
    cache = nv().PagedKV(k, v, dev.page_table, dev.k_scale, dev.v_scale)
    out, obig = guarded(torch.full(q.shape, 7.0, dtype=BF16), 3, 9.0)
    need = nv().lib.nvfp4_paged_attention_workspace_size(5, 0, 2, Hq, 2, 128, 2)
    ws, wbig = guarded(torch.zeros(need, dtype=torch.uint8), 4096, 0xA5)
    n, c = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (kv_len, cu))
    _, lse = nv().paged_attention(guarded(q, 3, float("nan"))[0], cache, n, c, out=out, workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    b.kv = kv
    want, want_lse, tol, tol_lse = b.attention()
    m = sum(new)
    assert_close(out[:m], want[:m], tol[:m])
    assert_close(lse[:m], want_lse[:m], tol_lse[:m])
    assert (out[m:] == 7.0).all() and edges_kept(obig, 3, 9.0) and edges_kept(wbig, 4096, 0xA5)
    assert edges_kept(kbig, 2, 0x7F) and edges_kept(vbig, 2, 0x7F)


@pytest.mark.parametrize("kv_len,cu,stores", [
    ([10 ** 9, -5], [0, 3, 5], {}),                            # past the table, before place 0
    ([2 ** 31 - 1, -2 ** 31], [0, 3, 5], {}),
    ([48, 33], [0, 10 ** 9, 5], {}),                           # every place before 0
    ([40, 33], [-4, 3, 3], {0: (0, 37), 1: (0, 38), 2: (0, 39)}),
    ([40, 33], [0, 3, 2 ** 31 - 1], {0: (0, 37), 1: (0, 38), 2: (0, 39)}),
])
def test_append_of_lengths_out_of_range(kv_len, cu, stores):
    b = Batch([3, 2], [48, 48], 8, 2, 128, True, seed=11)
    dev, _, _, q = b.device()
    k, kbig = guarded(b.k, 2, 0x55)
    v, vbig = guarded(b.v, 2, 0x55)
    cache = nv().PagedKV(k, v, dev.page_table, dev.k_scale, dev.v_scale)
    x = torch.randn(5, 2, 128, generator=torch.Generator().manual_seed(2)).to(BF16)
    q_out, qbig = guarded(torch.full(q.shape, 7.0, dtype=BF16), 3, 9.0)
    n, c = (torch.tensor(y, dtype=torch.int32, device=DEV) for y in (kv_len, cu))
    nv().kv_append(cache, gpu(x), gpu(x), n, c, q=q, q_out=q_out)
    torch.cuda.synchronize()
    codes = nv().fp8_kv_quantize(gpu(x), cache.k_scale), nv().fp8_kv_quantize(gpu(x), cache.v_scale)
    want = b.k.to(DEV), b.v.to(DEV)
    for t, (s, at) in stores.items():
        for w, code in zip(want, codes):
            w[int(b.table[s, at // 16]), :, at % 16] = code[t]
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert edges_kept(kbig, 2, 0x55) and edges_kept(vbig, 2, 0x55) and edges_kept(qbig, 3, 9.0)


# ---- calls around the operators -------------------------------------------------------------------------------------


def test_workspace_of_no_bytes_and_a_one_head_cache_of_either_layout():
    b = Batch([1] * 1100, [1 + (7 * i) % 50 for i in range(1100)], 2, 1, 64, True, seed=9)
    kv, kv_len, cu, q = b.device()
    assert nv().lib.nvfp4_paged_attention_workspace_size(1100, 1, 1100, 2, 1, 64, 2) == 0
    want = nv().paged_attention(q, kv, kv_len, cu, max_q=1)
    ws = torch.empty(0, dtype=torch.uint8, device=DEV)
    assert torch.equal(nv().paged_attention(q, kv, kv_len, cu, max_q=1, workspace=ws), want)
    flat = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kv.k, kv.v)]          # [pages, page_size, 1, dim]
    for x, y in zip(flat, (kv.k, kv.v)):
        assert torch.equal(x, y)
        x.as_strided_(x.shape, (16 * 64, 64, 64, 1))
    other = nv().PagedKV(*flat, kv.page_table, kv.k_scale, kv.v_scale)
    assert torch.equal(nv().paged_attention(q, other, kv_len, cu, max_q=1), want)


def test_layer_output_through_the_quantized_projection_by_value():
    a = Layer(2, 8, 2, 128, True, 16, 64, seed=3)
    new = [20, 1]
    a.len = [20, 1]
    kv_len, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (a.len, [0, 20, 21]))
    q, out = a.step(a.inputs(new).to(DEV), kv_len, cu)
    a.check(new, q, out)
    x = torch.randn(256, 1024, generator=torch.Generator().manual_seed(4)).to(BF16)
    w, act = nv().quantize(gpu(x)), nv().quantize(out.flatten(1), "per_row")
    assert_quant_equal(w, ref.quantize(x.float().numpy()), what="weights")
    assert_quant_equal(act, ref.quantize(out.flatten(1).float().cpu().numpy(), ref.PER_ROW), what="activations")
    Y, T = ref.gemm(to_host(act), to_host(w))
    assert_gemm_close(nv().gemm(act, w, F32), Y, T)

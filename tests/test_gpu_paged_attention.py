"""Attention over the paged cache against the plain 64-bit implementation: cache types, head layouts, single
tokens, drafts, chunks and whole prompts, windows, ragged and padded batches, pages that end inside a
tile, missing pages, rows that see nothing, non-finite values in places a row does not see."""
import pytest
import torch

from tests.gpu_helpers import DEV, nv
from tests.paged_helpers import Batch, assert_close

pytestmark = pytest.mark.gpu


def check(b: Batch, what="", scale=None, causal=True, window=0, max_q=0, **kw):
    kv, kv_len, cu, q = b.device()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    _, lse = nv().paged_attention(q, kv, kv_len, cu, scale=scale, causal=causal, window=window, max_q=max_q, out=out,
                                  return_lse=True, **kw)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = b.attention(scale, causal, window)
    c0, c1 = int(b.cu[0]), int(b.cu[-1])
    own = slice(c0, c1)
    assert_close(out[own], want[own], tol[own], what + " out")
    assert_close(lse[own], want_lse[own], tol_lse[own], what + " lse")
    assert (out[:c0] == 7.0).all() and (out[c1:] == 7.0).all(), "rows that belong to nobody were written"
    return out, lse


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(40, 8), (5, 1), (4, 4), (24, 1)])
def test_single_tokens(fp8, D, Hq, Hk):
    check(Batch([1] * 5, [1, 15, 16, 129, 700], Hq, Hk, D, fp8, seed=D + Hq), max_q=1)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 37])
def test_chunks_and_single_tokens_mixed(fp8, D, window):
    check(Batch([70, 1, 0, 3, 130, 1], [70, 33, 5, 200, 333, 600], 10, 2, D, fp8, seed=D, lead=2, tail=5), window=window)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("joint", [True, False])
def test_page_sizes_and_one_allocation(page, joint):
    check(Batch([1, 90, 2], [page + 1, 2 * page + 90, 3 * page - 1], 8, 2, 128, True, page=page, joint=joint, seed=page))


@pytest.mark.parametrize("n,L", [(1, 5000), (3, 4097), (6, 3001), (20, 2500), (200, 1999), (700, 700)])
@pytest.mark.parametrize("fp8", [True, False])
def test_one_sequence_split_over_workgroups(n, L, fp8):
    check(Batch([n], [L], 10, 2, 128, fp8, seed=n))


@pytest.mark.parametrize("fp8,D", [(True, 64), (False, 128), (True, 256), (False, 256)])
def test_drafts_two_row_blocks(fp8, D):
    check(Batch([4] * 6, [4, 9, 130, 257, 513, 1000], 28, 4, D, fp8, seed=5), max_q=4)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("n", [1, 40])
def test_no_causal_mask(fp8, n):
    check(Batch([n, n], [77, 300], 12, 3, 128, fp8, seed=n), causal=False)


def test_rows_that_see_nothing():
    # more new tokens than the cache holds, an empty cache, no new tokens
    check(Batch([9, 4, 0, 150, 1], [5, 0, 40, 20, 0], 10, 2, 128, True, seed=3))
    check(Batch([9, 4, 0, 150, 1], [5, 0, 40, 20, 0], 10, 2, 128, False, seed=3), causal=False)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("n", [1, 3, 100])
def test_missing_pages(fp8, n):
    b = Batch([n, n], [300, 333], 8, 2, 128, fp8, seed=n)
    b.table[0, 2] = -1
    b.table[0, 7] = b.k.shape[0]
    b.table[1, ::2] = 2 ** 31 - 1
    check(b)
    b.table[0, :] = -1                       # no page at all: zeros
    check(b)


def test_window_over_freed_pages():
    # pages before every row's window have been given back
    b = Batch([2, 60], [500, 700], 8, 2, 128, True, seed=8)
    b.table[0, :(500 - 2 - 100) // 16] = -1
    b.table[1, :(700 - 60 - 100) // 16] = -1
    check(b, window=100)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [4, 100])
def test_non_finite_values_reach_only_rows_that_see_them(fp8, D, n):
    b = Batch([n, n], [n + 50, 2 * n + 33], 8, 2, D, fp8, seed=n + D)
    for s in range(2):
        for back, d, val in ((n // 2, 3, "nan"), (1, 7, "inf"), (n - 1, 9, "-inf"), (n - 1, D - 1, "nan")):
            at = b.kv[s] - back
            p, r = int(b.table[s, at // 16]), at % 16
            if fp8:
                b.v[p, 1, r, d] = 0x7F if back % 2 else 0xFF
            else:
                b.v[p, 1, r, d] = float(val)
    check(b)


def test_non_finite_keys_a_row_does_not_see():
    b = Batch([40], [90], 8, 2, 128, False, seed=1)
    at = 89
    b.k[int(b.table[0, at // 16]), 0, at % 16, 5] = float("inf")
    b.q[:, :, 5] = b.q[:, :, 5].abs() + 1
    kv, kv_len, cu, q = b.device()
    out = nv().paged_attention(q, kv, kv_len, cu).float().cpu()
    want, _, tol, _ = b.attention()
    assert_close(out[:39], want[:39], tol[:39])
    assert torch.isnan(out[39, :4]).all()         # its score is +inf: inf - inf
    assert_close(out[39, 4:], want[39, 4:], tol[39, 4:])


def test_per_head_scales_and_scale_argument():
    check(Batch([1, 50], [300, 222], 12, 3, 128, True, per_head=True, seed=2), scale=0.03)
    check(Batch([1, 50], [300, 222], 12, 3, 64, True, per_head=True, seed=2), scale=1.7)   # peaked rows


def test_large_scores_move_the_running_maximum():
    # keys grow along the sequence, so the maximum keeps rising past the lazy threshold
    b = Batch([1, 64], [900, 700], 8, 2, 128, False, seed=6)
    for s in range(2):
        for at in range(b.kv[s]):
            b.k[int(b.table[s, at // 16]), :, at % 16] *= 0.01 + 6.0 * at / b.kv[s]
    check(b)
    b.k.mul_(-1)
    check(b)


def test_strided_queries_and_outputs():
    b = Batch([3, 80], [100, 150], 8, 2, 128, True, seed=4)
    kv, kv_len, cu, q = b.device()
    fused = torch.full((b.T, 8 * 128 + 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    view = fused[:, 256:256 + 1024].unflatten(1, (8, 128))
    view.copy_(q)
    wide = torch.full((b.T, 9, 136), 3.0, dtype=torch.bfloat16, device=DEV)
    nv().paged_attention(view, kv, kv_len, cu, out=wide[:, :8, :128])
    want = nv().paged_attention(q, kv, kv_len, cu)
    assert torch.equal(wide[:, :8, :128], want)
    assert (wide[:, 8] == 3.0).all() and (wide[:, :, 128:] == 3.0).all()
    heads_first = torch.empty((8, b.T, 128), dtype=torch.bfloat16, device=DEV)
    nv().paged_attention(q.transpose(0, 1).contiguous().transpose(0, 1), kv, kv_len, cu, out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), want)


@pytest.mark.parametrize("max_q", [0, 1, 2, 1000])
def test_the_hint_changes_no_result_beyond_rounding(max_q):
    check(Batch([1, 5, 64], [700, 333, 129], 10, 2, 128, True, seed=7), max_q=max_q)


def test_more_sequences_than_a_split_plans():
    new = [1] * 1100
    check(Batch(new, [1 + (7 * i) % 50 for i in range(1100)], 2, 1, 64, True, seed=9), max_q=1)


def test_same_bits_every_time_and_any_workspace_contents():
    b = Batch([1, 1, 40, 300], [4000, 17, 900, 1500], 10, 2, 128, True, seed=10)
    kv, kv_len, cu, q = b.device()
    need = nv().lib.nvfp4_paged_attention_workspace_size(b.T, 0, 4, 10, 2, 128, 2)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    ref = None
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out, lse = nv().paged_attention(q, kv, kv_len, cu, workspace=ws, return_lse=True)
        ref = (out.clone(), lse.clone()) if ref is None else ref
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_lengths_on_the_device_beyond_the_operands_are_clamped():
    b = Batch([3, 2], [40, 33], 8, 2, 128, True, seed=11)
    kv, _, _, q = b.device()
    for kv_len, cu in (([10 ** 9, -5], [0, 3, 5]), ([40, 33], [0, 10 ** 9, 5]), ([40, 33], [-4, 3, 2]), ([2 ** 31 - 1] * 2, [5, 0, 5])):
        out, lse = nv().paged_attention(q, kv, torch.tensor(kv_len, dtype=torch.int32, device=DEV),
                                        torch.tensor(cu, dtype=torch.int32, device=DEV), return_lse=True)
        torch.cuda.synchronize()


def test_cache_beyond_4_gb():
    # pages whose byte offsets pass 32 bits
    D, Hk, page = 128, 8, 64
    P = (5 << 30) // (Hk * page * D) + 1
    small = Batch([1, 70], [300, 200], 16, Hk, D, True, page=page, seed=12)
    kv, kv_len, cu, q = small.device()
    k = torch.empty((P, Hk, page, D), dtype=torch.uint8, device=DEV)
    v = torch.empty_like(k)
    n = small.k.shape[0]
    k[P - n:], v[P - n:] = kv.k, kv.v
    table = torch.where(kv.page_table >= 0, kv.page_table + (P - n), kv.page_table)
    big = nv().PagedKV(k, v, table, kv.k_scale, kv.v_scale)
    assert torch.equal(nv().paged_attention(q, big, kv_len, cu), nv().paged_attention(q, kv, kv_len, cu))


def test_no_tokens_and_no_sequences():
    b = Batch([1], [20], 8, 2, 128, True)
    kv, kv_len, cu, q = b.device()
    assert nv().paged_attention(q[:0], kv, kv_len, torch.zeros(2, dtype=torch.int32, device=DEV)).shape == (0, 8, 128)
    none = nv().PagedKV(kv.k, kv.v, kv.page_table[:0], kv.k_scale, kv.v_scale)
    out = torch.full_like(q, 2.0)
    nv().paged_attention(q, none, kv_len[:0], cu[:1], out=out)
    assert (out == 2.0).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    g = torch.Generator().manual_seed(100 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    Hk = r(1, 5)
    G = [1, 2, 3, 5, 8, 17, 33][r(0, 6)]
    S = r(1, 6)
    new = [[0, 1, 1, 2, 7, 33, 150][r(0, 6)] for _ in range(S)]
    new[0] = max(new[0], 1)
    kv = [max(0, n + [-3, 0, 1, 100, 777][r(0, 4)]) for n in new]
    b = Batch(new, kv, Hk * G, Hk, [64, 128, 256][r(0, 2)], bool(r(0, 1)), page=[16, 32, 128][r(0, 2)], seed=seed, tail=r(0, 3),
              per_head=bool(r(0, 1)))
    check(b, f"seed {seed}", window=[0, 0, 20, 200][r(0, 3)], max_q=[0, max(new)][r(0, 1)])

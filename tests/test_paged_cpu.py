"""Argument checks of the paged-cache operators, without a GPU: at the C ABI every malformed call returns
its status before any HIP call (pointers are fake addresses, never dereferenced), and the binding raises
ValueError before the library is called."""
import ctypes

import pytest
import torch

A16, MIS = 0x10000, 0x10001


@pytest.fixture(scope="module")
def nv():
    import nvfp4_w4a4_block_amd as m
    return m


def heads(nv, data=A16, n=8, tok=1024, head=128):
    return nv._Heads(data, n, tok, head)


def cache(nv, **kw):
    a = dict(k=A16, v=A16, num_pages=10, k_page_stride=2 * 16 * 128, v_page_stride=2 * 16 * 128, page_table=A16, table_stride=4,
             k_scale=A16, v_scale=A16, cu_q=A16, kv_len=A16, dtype=2, kv_heads=2, head_dim=128, page_size=16, num_seqs=3,
             table_width=4, scale_count=1)
    a.update(kw)
    return nv._PagedKV(**a)


BAD_CACHES = [(dict(k=None), 1), (dict(v=MIS), 1), (dict(num_pages=0), 1), (dict(k_page_stride=100), 1),
              (dict(v_page_stride=2 * 16 * 128 + 8), 1), (dict(page_table=None), 1), (dict(table_stride=3), 1), (dict(k_scale=None), 1),
              (dict(v_scale=MIS), 1), (dict(scale_count=3), 1), (dict(scale_count=0), 1), (dict(cu_q=None), 1), (dict(kv_len=MIS), 1),
              (dict(dtype=0), 1), (dict(dtype=9), 1), (dict(kv_heads=0), 1), (dict(page_size=24), 1), (dict(page_size=0), 1),
              (dict(page_size=8), 2), (dict(page_size=2048), 2), (dict(num_seqs=-1), 1), (dict(table_width=1 << 28), 2),
              (dict(num_pages=1 << 31), 2)]


def attend(nv, c=None, T=5, max_q=0, q=True, scale=0.1, causal=1, window=0, out=True, lse=None, ws=A16, wsb=1 << 40):
    q = heads(nv) if q is True else q
    out = heads(nv) if out is True else out
    return nv.lib.nvfp4_paged_attention(cache(nv) if c is None else c, T, max_q, q, scale, causal, window, out, lse, ws, wsb, None)


def test_attention_argument_errors(nv):
    for kw, status in BAD_CACHES:
        assert attend(nv, cache(nv, **kw)) == status, kw
    assert nv.lib.nvfp4_paged_attention(None, 5, 0, heads(nv), 0.1, 1, 0, heads(nv), None, A16, 1 << 40, None) == 1
    assert attend(nv, T=-1) == 1 and attend(nv, max_q=-1) == 1
    assert attend(nv, q=None) == 1 and attend(nv, out=None) == 1
    assert attend(nv, q=heads(nv, MIS)) == 1 and attend(nv, q=heads(nv, None)) == 1
    assert attend(nv, q=heads(nv, n=7)) == 1 and attend(nv, q=heads(nv, n=0)) == 1       # not a multiple of the cache's heads
    assert attend(nv, q=heads(nv, n=10)) == 1                                             # not the output's heads
    assert attend(nv, q=heads(nv, tok=1025)) == 1 and attend(nv, q=heads(nv, head=64)) == 1
    assert attend(nv, out=heads(nv, tok=512)) == 1 and attend(nv, out=heads(nv, tok=0)) == 1   # overlapping output rows
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attend(nv, scale=scale) == 1
    assert attend(nv, causal=2) == 1 and attend(nv, window=-1) == 1 and attend(nv, causal=0, window=5) == 1
    assert attend(nv, lse=0x10002) == 1
    assert attend(nv, ws=None) == 3 and attend(nv, wsb=16) == 3 and attend(nv, ws=A16 + 8) == 3
    for d in (16, 96, 512):
        assert attend(nv, cache(nv, head_dim=d, k_page_stride=1 << 20, v_page_stride=1 << 20), q=heads(nv, head=512, tok=4096),
                      out=heads(nv, head=512, tok=4096)) == 2
    assert attend(nv, cache(nv, kv_heads=1), q=heads(nv, n=257, tok=1 << 20), out=heads(nv, n=257, tok=1 << 20)) == 2
    assert attend(nv, T=0) == 0 and attend(nv, cache(nv, num_seqs=0)) == 0                # nothing to do


def test_attention_workspace_size(nv):
    size = nv.lib.nvfp4_paged_attention_workspace_size
    assert size(1, 1, 1, 40, 8, 128, 2) > 0
    assert size(0, 1, 1, 40, 8, 128, 2) == 0 and size(1, 1, 1, 40, 7, 128, 2) == 0 and size(1, 1, 1, 40, 8, 96, 2) == 0
    assert size(1, 1, 1, 40, 8, 128, 0) == 0 and size(1, -1, 1, 40, 8, 128, 2) == 0
    # enough row tiles to fill the GPU: nothing is split, nothing needed
    assert size(1 << 20, 1 << 20, 1, 40, 8, 128, 2) == 0


def rope(nv, table=A16, rows=64, pos=A16, dim=128, inter=0):
    return nv._Rope(table, rows, pos, dim, inter)


BAD_ROPES = [dict(table=None), dict(table=A16 + 8), dict(rows=-1), dict(pos=0x10002), dict(dim=0), dict(dim=24), dict(dim=144),
             dict(inter=2)]


def test_norm_rope_argument_errors(nv):
    def f(T=5, D=128, xt=1, q=True, k=None, qw=None, kw=None, eps=1e-6, r=None, ot=1, qo=True, ko=None):
        q, qo = (heads(nv) if x is True else x for x in (q, qo))
        return nv.lib.nvfp4_qk_norm_rope(T, D, xt, q, k, qw, kw, eps, r, ot, qo, ko, None)
    assert f(T=-1) == 1 and f(D=0) == 1 and f(D=24) == 1 and f(D=528) == 2 and f(xt=2) == 1 and f(ot=7) == 1
    assert f(q=None) == 1 and f(qo=None) == 1 and f(k=heads(nv)) == 1 and f(ko=heads(nv)) == 1
    assert f(q=heads(nv, MIS)) == 1 and f(qo=heads(nv, n=7)) == 1 and f(k=heads(nv, n=2), ko=heads(nv, n=3)) == 1
    assert f(qo=heads(nv, tok=0)) == 1 and f(q=heads(nv, tok=1028)) == 1
    assert f(qw=0x10004) == 1 and f(kw=0x10004, k=heads(nv), ko=heads(nv)) == 1
    assert f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    for kw in BAD_ROPES:
        assert f(r=rope(nv, **kw)) == 1, kw
    assert f(r=rope(nv, pos=None)) == 1
    assert f(T=0) == 0


def test_append_argument_errors(nv):
    def kh(**kw):
        return heads(nv, n=kw.pop("n", 2), **kw)

    def f(c=None, T=5, xt=1, k=True, v=True, kw=None, eps=1e-6, r=None, q=None, qw=None, qt=1, qo=None):
        k, v = (kh() if x is True else x for x in (k, v))
        return nv.lib.nvfp4_kv_append(cache(nv) if c is None else c, T, xt, k, v, kw, eps, r, q, qw, qt, qo, None)
    for kw, status in BAD_CACHES:
        assert f(cache(nv, **kw)) == status, kw
    assert f(T=-1) == 1 and f(xt=2) == 1 and f(k=None) == 1 and f(v=None) == 1 and f(k=kh(n=3)) == 1 and f(v=kh(n=1)) == 1
    assert f(k=kh(data=MIS)) == 1 and f(v=kh(tok=1030)) == 1 and f(kw=0x10008) == 1 and f(eps=-1e-6) == 1
    assert f(q=heads(nv)) == 1 and f(qo=heads(nv)) == 1 and f(q=heads(nv), qo=heads(nv), qt=2) == 1
    assert f(q=heads(nv), qo=heads(nv, n=4)) == 1 and f(q=heads(nv), qo=heads(nv, tok=128)) == 1
    assert f(cache(nv, head_dim=24, k_page_stride=1 << 16, v_page_stride=1 << 16)) == 1
    assert f(cache(nv, head_dim=528, k_page_stride=1 << 16, v_page_stride=1 << 16)) == 2
    for kw in BAD_ROPES:
        assert f(r=rope(nv, **kw)) == 1, kw
    assert f(T=0) == 0 and f(cache(nv, num_seqs=0)) == 0


def batch(nv, fp8=True, D=64, Hk=2, pages=5, S=3, T=4, Hq=4):
    shape = (pages, Hk, 16, D)
    k = torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16)
    s = torch.ones(1) if fp8 else None
    kv = nv.PagedKV(k, k.clone(), torch.zeros(S, 4, dtype=torch.int32), s, s)
    return (kv, torch.zeros(S, dtype=torch.int32), torch.zeros(S + 1, dtype=torch.int32), torch.zeros(T, Hq, D, dtype=torch.bfloat16),
            torch.zeros(T, Hk, D, dtype=torch.bfloat16))


def test_binding_checks_the_cache(nv):
    kv, n, cu, q, k = batch(nv)
    with pytest.raises(ValueError, match="GPU"):
        nv.paged_attention(q, kv, n, cu)
    with pytest.raises(ValueError, match="GPU"):
        nv.kv_append(kv, k, k, n, cu)
    P = nv.PagedKV
    for bad, match in ((P(kv.k, kv.v[:3], kv.page_table, kv.k_scale, kv.v_scale), "one shape"),
                       (P(kv.k[0], kv.v[0], kv.page_table, kv.k_scale, kv.v_scale), "one shape"),
                       (P(kv.k.int(), kv.v.int(), kv.page_table, kv.k_scale, kv.v_scale), "uint8"),
                       (P(kv.k.transpose(1, 2), kv.v.transpose(1, 2), kv.page_table, kv.k_scale, kv.v_scale), "contiguous"),
                       (P(kv.k, kv.v, kv.page_table.long(), kv.k_scale, kv.v_scale), "page_table"),
                       (P(kv.k, kv.v, kv.page_table.T.contiguous().T, kv.k_scale, kv.v_scale), "page_table"),
                       (P(kv.k, kv.v, kv.page_table), "calibrated"),
                       (P(kv.k, kv.v, kv.page_table, torch.ones(3), torch.ones(3)), "k_scale"),
                       (P(kv.k, kv.v, kv.page_table, torch.ones(2), torch.ones(1)), "v_scale"),
                       (P(kv.k, kv.v, kv.page_table, torch.ones(1).double(), torch.ones(1)), "k_scale")):
        with pytest.raises(ValueError, match=match):
            nv.paged_attention(q, bad, n, cu)
        with pytest.raises(ValueError, match=match):
            nv.kv_append(bad, k, k, n, cu)
    for a, b, match in ((n.long(), cu, "kv_len"), (n[:2], cu, "kv_len"), (n, cu[:3], "cu_q"), (n, cu.float(), "cu_q"),
                        (n[:, None], cu, "kv_len")):
        with pytest.raises(ValueError, match=match):
            nv.paged_attention(q, kv, a, b)
    with pytest.raises(ValueError, match="PagedKV"):
        nv.paged_attention(q, (kv.k, kv.v), n, cu)


def test_binding_checks_operands(nv):
    kv, n, cu, q, k = batch(nv)
    for bad, match in ((q[0], "q"), (q.float(), "dtype"), (q[:, :3], "multiple"), (torch.zeros(4, 4, 32, dtype=torch.bfloat16), "shape"),
                       (q.transpose(1, 2).contiguous().transpose(1, 2), "contiguous")):
        with pytest.raises(ValueError, match=match):
            nv.paged_attention(bad, kv, n, cu)
    with pytest.raises(ValueError, match="out"):
        nv.paged_attention(q, kv, n, cu, out=q[:2])
    with pytest.raises(ValueError, match="out"):
        nv.paged_attention(q, kv, n, cu, out=q.float())
    with pytest.raises(ValueError, match="workspace"):
        nv.paged_attention(q, kv, n, cu, workspace=torch.zeros(4))
    with pytest.raises(ValueError, match="v:"):
        nv.kv_append(kv, k, k.float(), n, cu)
    with pytest.raises(ValueError, match="k:"):
        nv.kv_append(kv, k[:, :1], k, n, cu)
    with pytest.raises(ValueError, match="without q"):
        nv.kv_append(kv, k, k, n, cu, q_weight=torch.ones(64))
    with pytest.raises(ValueError, match="k_weight"):
        nv.kv_append(kv, k, k, n, cu, k_weight=torch.ones(32))
    with pytest.raises(ValueError, match="q:"):
        nv.kv_append(kv, k, k, n, cu, q=q.float())
    with pytest.raises(ValueError, match="positions"):
        nv.kv_append(kv, k, k, n, cu, positions=n)
    with pytest.raises(ValueError, match="positions"):
        nv.kv_append(kv, k, k, n, cu, rope=torch.zeros(9, 64), positions=n)
    with pytest.raises(ValueError, match="rope"):
        nv.kv_append(kv, k, k, n, cu, rope=torch.zeros(9, 64).double())
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        nv.qk_norm_rope(q, k, rope=torch.zeros(9, 64), positions=pos)
    with pytest.raises(ValueError, match="positions"):
        nv.qk_norm_rope(q, k, rope=torch.zeros(9, 64))
    with pytest.raises(ValueError, match="without k"):
        nv.qk_norm_rope(q, k_weight=torch.ones(64))
    with pytest.raises(ValueError, match="dtype"):
        nv.qk_norm_rope(q.half())
    with pytest.raises(ValueError, match="out_dtype"):
        nv.qk_norm_rope(q, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="q_out"):
        nv.qk_norm_rope(q, q_out=q.float())
    with pytest.raises(ValueError, match="k:"):
        nv.qk_norm_rope(q, k[:3])


def test_structures_match_the_header(nv):
    # field offsets of the binding's structures follow the C layout rules of the header's
    assert ctypes.sizeof(nv._Heads) == 32 and ctypes.sizeof(nv._Rope) == 32 and ctypes.sizeof(nv._PagedKV) == 120

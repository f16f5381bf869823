"""Argument checks of the Gated DeltaNet layer's operators and the norms with quantized outputs, without a GPU: at the C
ABI every malformed call returns its status before any HIP call (pointers are fake addresses, never
dereferenced), and the binding raises ValueError before the library is called."""
import pytest
import torch

A16, MIS, INF, NAN = 0x10000, 0x10001, float("inf"), float("nan")


@pytest.fixture(scope="module")
def nv():
    import nvfp4_w4a4_block_amd as m
    return m


def heads(nv, data=A16, n=8, tok=1024, head=128):
    return nv._Heads(data, n, tok, head)


def norm_out(nv, **kw):
    a = dict(y=A16, ldy=64, codes=A16, block_scales=A16, scale=A16, y_dtype=1, format=1, mode=1)
    a.update(kw)
    return nv._NormOut(*a.values())


def states(nv, **kw):
    a = dict(data=A16, num_slots=4, slot_stride=1 << 22, slots=A16, cu_q=A16, kv_len=A16, num_seqs=3)
    a.update(kw)
    return nv._SeqStates(*a.values())


BAD_OUTS = [dict(format=3), dict(format=-1), dict(y=None, format=0), dict(y=MIS), dict(y_dtype=2), dict(ldy=48), dict(ldy=65),
            dict(mode=0), dict(mode=3), dict(codes=None), dict(codes=A16 + 8), dict(scale=None), dict(scale=MIS), dict(block_scales=None)]


def test_add_rms_norm_argument_errors(nv):
    def call(o=None, rows=3, cols=64, x=A16, xd=1, ldx=64, r=A16, rd=1, ldr=64, w=A16, eps=1e-6, ro=A16, ldro=64):
        return nv.lib.nvfp4_add_rms_norm(rows, cols, x, xd, ldx, r, rd, ldr, w, eps, ro, ldro, norm_out(nv) if o is None else o, None)
    for kw in BAD_OUTS:
        assert call(norm_out(nv, **kw)) == 1, kw
    assert nv.lib.nvfp4_add_rms_norm(3, 64, A16, 1, 64, None, 1, 0, A16, 1e-6, None, 0, None, None) == 1
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=40), dict(x=None), dict(x=MIS), dict(xd=2), dict(ldx=63), dict(ldx=68), dict(rd=2),
               dict(ldr=48), dict(r=A16 + 4), dict(w=None), dict(w=A16 + 4), dict(eps=-1.0), dict(eps=NAN), dict(ro=MIS), dict(ldro=63),
               dict(r=None)):
        assert call(**kw) == 1, kw
    assert call(cols=32784, ldx=1 << 16, ldr=1 << 16, ldro=1 << 16) == 2 and call(rows=1 << 21) == 2
    assert call(rows=0) == 0


def test_gated_rms_norm_argument_errors(nv):
    def call(o=None, T=3, D=128, x=True, xd=1, z=True, zd=1, w=A16, eps=1e-6):
        x, z = (heads(nv) if v is True else v for v in (x, z))
        return nv.lib.nvfp4_gated_rms_norm(T, D, x, xd, z, zd, w, eps, norm_out(nv, ldy=1024) if o is None else o, None)
    for kw in BAD_OUTS:
        assert call(norm_out(nv, **dict(dict(ldy=1024), **kw))) == 1, kw
    for kw in (dict(T=-1), dict(D=0), dict(D=8), dict(D=96), dict(x=None), dict(z=None), dict(x=heads(nv, None)), dict(z=heads(nv, MIS)),
               dict(z=heads(nv, n=4)), dict(x=heads(nv, head=64)), dict(z=heads(nv, tok=1025)), dict(xd=2), dict(zd=-1), dict(w=None),
               dict(w=A16 + 8), dict(eps=-1.0)):
        assert call(**kw) == 1, kw
    assert call(D=2048) == 2 and call(T=1 << 21) == 2
    assert call(x=heads(nv, n=257, tok=1 << 16), z=heads(nv, n=257, tok=1 << 16)) == 2
    assert call(T=0) == 0


BAD_STATES = [(dict(num_seqs=-1), 1), (dict(num_slots=-1), 1), (dict(num_slots=1 << 31), 2), (dict(cu_q=None), 1), (dict(cu_q=MIS), 1),
              (dict(kv_len=None), 1), (dict(slots=MIS), 1), (dict(data=None), 1), (dict(data=A16 + 8), 1), (dict(slot_stride=64), 1),
              (dict(slot_stride=(1 << 22) + 1), 1)]


def test_gdn_conv_argument_errors(nv):
    def call(s=None, T=5, C=64, W=4, x=A16, xd=1, ldx=64, w=A16, b=A16, y=A16, yd=1, ldy=64):
        return nv.lib.nvfp4_gdn_conv(states(nv) if s is None else s, T, C, W, x, xd, ldx, w, b, y, yd, ldy, None)
    for kw, status in BAD_STATES:
        assert call(states(nv, **kw)) == status, kw
    for kw in (dict(T=-1), dict(C=0), dict(C=60), dict(x=None), dict(x=MIS), dict(xd=2), dict(ldx=56), dict(ldx=65), dict(w=None), dict(w=MIS),
               dict(b=MIS), dict(y=None), dict(y=MIS), dict(yd=2), dict(ldy=56), dict(ldy=68)):
        assert call(**kw) == 1, kw
    assert nv.lib.nvfp4_gdn_conv(None, 5, 64, 4, A16, 1, 64, A16, None, A16, 1, 64, None) == 1
    assert call(W=1) == 2 and call(W=5) == 2 and call(T=1 << 30) == 2 and call(C=(1 << 24) + 8) == 2
    assert call(T=0) == 0 and call(states(nv, num_seqs=0, cu_q=None)) == 0


def test_gated_delta_rule_argument_errors(nv):
    def call(s=None, T=5, mq=0, dk=128, dv=128, q=True, k=True, v=True, g=A16, b=A16, scale=0.1, out=True, ws=A16, wsb=1 << 40):
        q, k, v, out = (heads(nv) if t is True else t for t in (q, k, v, out))
        return nv.lib.nvfp4_gated_delta_rule(states(nv) if s is None else s, T, mq, dk, dv, q, k, v, g, b, scale, out, ws, wsb, None)
    for kw, status in BAD_STATES:
        assert call(states(nv, **kw)) == status, kw
    for kw in (dict(T=-1), dict(mq=-1), dict(dk=0), dict(dv=0), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=heads(nv, MIS)),
               dict(k=heads(nv, n=4)), dict(v=heads(nv, n=12), out=heads(nv, n=12)), dict(v=heads(nv, n=16)), dict(q=heads(nv, n=0), k=heads(nv, n=0)),
               dict(k=heads(nv, tok=1028)), dict(v=heads(nv, head=64)), dict(out=heads(nv, tok=512)), dict(g=None), dict(b=None), dict(g=MIS),
               dict(b=MIS), dict(scale=INF), dict(scale=NAN)):
        assert call(**kw) == 1, kw
    for kw in (dict(dk=32), dict(dk=96), dict(dk=256), dict(dv=48), dict(dv=544), dict(T=1 << 30)):
        assert call(**kw) == 2, kw
    assert call(v=heads(nv, tok=1 << 24)) == 2 and call(out=heads(nv, tok=1 << 24)) == 2
    assert call(T=0) == 0 and call(states(nv, num_seqs=0, cu_q=None)) == 0
    assert nv.lib.nvfp4_gated_delta_rule(None, 5, 0, 128, 128, heads(nv), heads(nv), heads(nv), A16, A16, 0.1, heads(nv), A16, 1 << 40, None) == 1


def bad(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_refusals_norms(nv):
    x, w = torch.zeros(3, 64), torch.ones(64)
    for kw, match in ((dict(x=torch.zeros(3)), "x:"), (dict(x=x.half()), "dtype"), (dict(x=torch.zeros(64, 3).T), "contiguous"),
                      (dict(weight=w.bfloat16()), "weight"), (dict(weight=w[:32]), "weight"), (dict(residual=x[:2]), "residual"),
                      (dict(residual=x.half()), "residual"), (dict(residual_out=x), "residual_out"), (dict(out_dtype=torch.float16), "out_dtype"),
                      (dict(out_dtype=None), "ask for"), (dict(quant="int8"), "quant"), (dict(quant="fp8", mode="per_tensor"), "mode"),
                      (dict(quant="fp8", mode="given"), "needs scale"), (dict(quant="fp8", scale=w[:1]), "scale"), (dict(scale=w[:1]), "scale"),
                      (dict(quant="fp8", mode="given", scale=w[:2]), "scale"), (dict(out=x), "out"),
                      (dict(quant="nvfp4", q_out=nv.FP8Tensor(x, w)), "q_out"),
                      (dict(residual=x, residual_out=x.bfloat16()), "residual_out"), (dict(), "GPU")):
        bad(match, nv.add_rms_norm, **{"x": x, "weight": w, **kw})
    bad("multiple of 16", nv.add_rms_norm, torch.zeros(3, 40), torch.ones(40), quant="fp8")
    h, w = torch.zeros(3, 2, 64), torch.ones(64)
    for kw, match in ((dict(x=x), "x:"), (dict(z=torch.zeros(3, 2, 32)), "z:"), (dict(z=h.half()), "z:"), (dict(weight=torch.ones(128)), "weight"),
                      (dict(out_dtype=None), "ask for"), (dict(), "GPU")):
        bad(match, nv.gated_rms_norm, **{"x": h, "z": h, "weight": w, **kw})


def test_binding_refusals_sequences(nv):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x, w, pool = torch.zeros(5, 64), torch.zeros(64, 4), torch.zeros(4, 3, 64)
    base = dict(state=nv.GDNState(i32(2, 0), conv=pool), x=x, weight=w, kv_len=i32(3, 2), cu_q=i32(0, 3, 5))
    for kw, match in ((dict(state=pool), "GDNState"), (dict(state=nv.GDNState()), "state.conv"), (dict(state=nv.GDNState(conv=pool[:, :2])), "state.conv"),
                      (dict(state=nv.GDNState(conv=pool.bfloat16())), "state.conv"), (dict(state=nv.GDNState(conv=torch.zeros(3, 4, 64).transpose(0, 1))), "contiguous"),
                      (dict(state=nv.GDNState(i32(1), conv=pool)), "slots"), (dict(kv_len=i32(1)), "kv_len"), (dict(cu_q=i32(0, 3, 5).long()), "cu_q"),
                      (dict(weight=w.T), "weight"), (dict(weight=torch.zeros(64, 5)), "width"), (dict(weight=w.bfloat16()), "weight"),
                      (dict(bias=torch.zeros(3)), "bias"), (dict(x=x.half()), "dtype"), (dict(out=x), "out"), (dict(out_dtype=torch.half), "out_dtype"),
                      (dict(), "GPU")):
        bad(match, nv.gdn_conv, **{**base, **kw})
    bf = torch.bfloat16
    q, v, g, pool = torch.zeros(5, 2, 64, dtype=bf), torch.zeros(5, 4, 32, dtype=bf), torch.zeros(5, 4), torch.zeros(4, 4, 64, 32)
    base = dict(state=nv.GDNState(i32(2, 0), delta=pool), q=q, k=q, v=v, g=g, beta=g, kv_len=i32(3, 2), cu_q=i32(0, 3, 5))
    for kw, match in ((dict(state=pool), "GDNState"), (dict(state=nv.GDNState()), "state.delta"), (dict(state=nv.GDNState(delta=pool[:, :2])), "state.delta"),
                      (dict(state=nv.GDNState(delta=pool.bfloat16())), "state.delta"), (dict(state=nv.GDNState(delta=torch.zeros(4, 4, 32, 64).transpose(2, 3))), "contiguous"),
                      (dict(q=q.float()), "q:"), (dict(k=q[:, :1]), "k:"), (dict(v=v.float()), "v:"), (dict(v=torch.zeros(5, 3, 32, dtype=bf)), "multiple"),
                      (dict(g=g.bfloat16()), "g:"), (dict(beta=g[:, :2]), "beta"), (dict(g=torch.zeros(5, 8)[:, :4]), "g:"), (dict(kv_len=i32(1)), "kv_len"),
                      (dict(cu_q=g), "cu_q"), (dict(out=v.float()), "out"), (dict(workspace=g), "workspace"), (dict(), "GPU")):
        bad(match, nv.gated_delta_rule, **{**base, **kw})


def test_gated_delta_rule_workspace(nv):
    size = nv.lib.nvfp4_gated_delta_rule_workspace_size
    need = size(100, 0, 2, 8, 8, 128, 128)
    assert need > 0 and need % 16 == 0
    # single tokens and drafts need none; a hint past them does, and more tokens and sequences need more
    assert size(16, 0, 2, 8, 8, 128, 128) == size(100, 16, 8, 8, 8, 128, 128) == 0
    assert size(100, 17, 2, 8, 8, 128, 128) == need < size(164, 0, 2, 8, 8, 128, 128) < size(164, 0, 3, 8, 8, 128, 128)
    for args in ((-1, 0, 2, 8, 8, 128, 128), (100, -1, 2, 8, 8, 128, 128), (100, 0, 0, 8, 8, 128, 128), (100, 0, 2, 0, 8, 128, 128),
                 (100, 0, 2, 8, 12, 128, 128), (100, 0, 2, 8, 8, 96, 128), (100, 0, 2, 8, 8, 128, 48), (100, 0, 2, 8, 8, 128, 544),
                 (1 << 30, 0, 2, 8, 8, 128, 128)):
        assert size(*args) == 0, args

    def call(ws, wsb):
        return nv.lib.nvfp4_gated_delta_rule(states(nv), 100, 0, 128, 128, heads(nv), heads(nv), heads(nv), A16, A16, 0.1, heads(nv), ws, wsb, None)
    need = size(100, 0, states(nv).num_seqs, 8, 8, 128, 128)
    assert call(None, need) == call(A16, need - 1) == call(A16, 0) == call(MIS, need) == 3


def test_launches_too_large_are_refused(nv):
    # 2^26 runs of 16 tokens: a thread more than a launch can have
    assert nv.lib.nvfp4_gdn_conv(states(nv), (1 << 30) - 1, 8, 4, A16, nv._BF16, 8, A16, None, A16, nv._BF16, 8, None) == 2
    assert nv.lib.nvfp4_gdn_conv(states(nv, num_seqs=(1 << 31) - 1), 8, 8, 4, A16, nv._BF16, 8, A16, None, A16, nv._BF16, 8, None) == 2
    many = states(nv, num_seqs=1 << 24)
    assert nv.lib.nvfp4_gated_delta_rule(many, 1, 0, 128, 128, heads(nv), heads(nv), heads(nv), A16, A16, 0.1, heads(nv), None, 0, None) == 2


def test_binding_refuses_a_small_workspace(nv):
    bf = torch.bfloat16
    q, v, g = torch.zeros(50, 2, 64, dtype=bf), torch.zeros(50, 4, 32, dtype=bf), torch.zeros(50, 4)
    lens = torch.tensor([30, 20], dtype=torch.int32), torch.tensor([0, 30, 50], dtype=torch.int32)
    need = nv.lib.nvfp4_gated_delta_rule_workspace_size(50, 0, 2, 2, 4, 64, 32)
    for ws, match in ((torch.zeros(need - 1, dtype=torch.uint8), "needed"), (torch.zeros(2 * need, dtype=torch.uint8)[::2], "contiguous"),
                      (torch.zeros(need, dtype=torch.int8), "uint8")):
        bad(match, nv.gated_delta_rule, nv.GDNState(delta=torch.zeros(2, 4, 64, 32)), q, q, v, g, g, *lens, workspace=ws)

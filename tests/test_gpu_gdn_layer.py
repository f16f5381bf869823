"""A Gated DeltaNet layer's step as it is used: norm in front of the fused projection with its gates, convolution,
gated delta rule, gated norm, output projection, norm behind; prompts in chunks and single tokens in one batch, states
in a pool.  Every stage is checked against 64 bits from what it read; then the step captured, on several streams, with
a shared workspace, and operands past 32-bit offsets."""
import pytest
import torch

from oracle import nvfp4_ref as ref
from tests.gdn_helpers import BF16, F32, HALF, Seqs, add_norm, assert_within, conv, delta_inputs, delta_rule, gated_norm, rand
from tests.gpu_helpers import DEV, assert_quant_equal, nv

pytestmark = pytest.mark.gpu
EPS = 1e-6


class Layer:
    def __init__(self, seqs, hidden=256, Hk=4, Hv=8, D=128, W=4, seed=0):
        self.hidden, self.Hk, self.Hv, self.D, self.seed = hidden, Hk, Hv, D, seed
        self.C = 2 * Hk * D + Hv * D
        self.widths = [Hk * D, Hk * D, Hv * D, Hv * D, Hv, Hv]
        q = [nv().quantize(rand(n, hidden, seed=seed + 10 + i, scale=0.06).to(DEV)) for i, n in enumerate(self.widths)]
        self.w_in = torch.cat([x.codes for x in q]), torch.cat([x.scales for x in q]), torch.cat([x.global_scale for x in q])
        self.w_out = nv().quantize(rand(hidden, Hv * D, seed=seed + 20, scale=0.03).to(DEV))
        self.norm, self.head_norm = 1 + rand(hidden, seed=seed + 21, dtype=F32, scale=0.1), 1 + rand(D, seed=seed + 22, dtype=F32, scale=0.1)
        self.w_conv, self.bias = rand(self.C, W, seed=seed + 23, dtype=F32, scale=0.5), rand(self.C, seed=seed + 24, dtype=F32, scale=0.1)
        self.a_log, self.dt = rand(Hv, seed=seed + 25, dtype=F32).abs(), rand(Hv, seed=seed + 26, dtype=F32) - 3
        self.on_gpu = [x.to(DEV) for x in (self.norm, self.head_norm, self.w_conv, self.bias, self.a_log, self.dt)]
        num = seqs + 2
        self.state = nv().GDNState(torch.randperm(num, generator=torch.Generator().manual_seed(seed))[:seqs].to(torch.int32).to(DEV),
                                   torch.full((num, W - 1, self.C), float("nan"), dtype=BF16, device=DEV),
                                   torch.full((num, Hv, D, D), float("nan"), device=DEV))

    def copy_state(self):
        s = self.state
        return nv().GDNState(s.slots.clone(), s.conv.clone(), s.delta.clone())

    def step(self, h, residual, kv_len, cu_q, max_q=0, state=None, workspace=None):
        """Everything the step makes, in order."""
        state = self.state if state is None else state
        norm, head_norm, w_conv, bias, a_log, dt = self.on_gpu
        Hk, Hv, D, T = self.Hk, self.Hv, self.D, h.shape[0]
        _, a, r = nv().add_rms_norm(h, norm, residual, EPS, out_dtype=None, quant="nvfp4")
        p, g, beta = nv().gemm_fused_gdn_gates(a, self.w_in[0], self.w_in[1], self.widths, self.w_in[2], a_log, dt)
        x = nv().gdn_conv(state, p[:, :self.C], w_conv, kv_len, cu_q, bias, out=torch.zeros(T, self.C, dtype=BF16, device=DEV))
        q, k = x[:, :Hk * D].unflatten(1, (Hk, D)), x[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D))
        v, z = x[:, 2 * Hk * D:].unflatten(1, (Hv, D)), p[:, self.C:self.C + Hv * D].unflatten(1, (Hv, D))
        o = nv().gated_delta_rule(state, q, k, v, g, beta, kv_len, cu_q, max_q=max_q, workspace=workspace,
                                  out=torch.zeros(T, Hv, D, dtype=BF16, device=DEV))
        _, b = nv().gated_rms_norm(o, z, head_norm, EPS, out_dtype=None, quant="nvfp4")
        y = nv().gemm(b, self.w_out, BF16)
        return dict(h=h, residual=residual, a=a, r=r, p=p, g=g, beta=beta, x=x, q=q, k=k, v=v, z=z, o=o, b=b, y=y)

    def check(self, b: Seqs, before, m):
        """The stages of a step against 64 bits, each from the inputs that it had."""
        c = {n: t.cpu() if isinstance(t, torch.Tensor) else t for n, t in m.items()}
        r, y = add_norm(c["h"], c["residual"], self.norm, EPS)
        assert torch.equal(c["r"], r)
        assert_quant_equal(m["a"], ref.quantize(y.numpy(), ref.PER_ROW), what="norm in front")
        rows = b.rows()
        want, tol, states = conv(b, c["p"][:, :self.C], self.w_conv, self.bias, before.conv.cpu())
        assert_within(c["x"][rows], want[rows], tol[rows] + HALF[BF16] * want[rows].abs(), "convolution")
        used = b.slots[torch.tensor(b.new) > 0].long()
        assert torch.equal(self.state.conv.cpu()[used], states[used])
        o, o_tol, s, s_tol = delta_rule(b, c["q"], c["k"], c["v"], c["g"], c["beta"], before.delta.cpu())
        assert_within(c["o"][rows], o[rows], o_tol[rows], "delta rule")
        assert_within(self.state.delta.cpu(), s, s_tol, "states")
        y, _, _ = gated_norm(c["o"], c["z"], self.head_norm, EPS)
        assert_quant_equal(m["b"], ref.quantize(y.float().flatten(1).numpy(), ref.PER_ROW), what="gated norm")
        assert torch.isfinite(c["y"]).all() and (c["x"][~rows] == 0).all() and (c["o"][~rows] == 0).all()


def batch(layer, new, past, behind=0):
    b = Seqs(new, past, behind=behind)
    b.slots, b.num_slots = layer.state.slots.cpu(), layer.state.conv.shape[0]
    return b


@pytest.mark.parametrize("hint", [True, False])
def test_prompts_in_chunks_and_single_tokens_together(hint):
    a = Layer(4)
    past = [0, 0, 0, 0]
    for i, new in enumerate(([70, 3, 0, 1], [1, 1, 1, 1], [20, 0, 130, 1], [1, 1, 1, 1], [2, 65, 1, 0])):
        b = batch(a, new, past, behind=i)
        h, residual = rand(b.T, a.hidden, seed=30 + i).to(DEV), rand(b.T, a.hidden, seed=40 + i).to(DEV)
        before = a.copy_state()
        m = a.step(h, residual, *b.gpu(), max_q=max(new) if hint else 0)
        a.check(b, before, m)
        # the next layer's norm on what this one made
        y, q, r = nv().add_rms_norm(m["y"], a.on_gpu[0], m["r"], EPS, quant="nvfp4")
        want_r, want_y = add_norm(m["y"].cpu(), m["r"].cpu(), a.norm, EPS)
        assert torch.equal(r.cpu(), want_r) and torch.equal(y.cpu(), want_y.to(BF16))
        assert_quant_equal(q, ref.quantize(want_y.numpy(), ref.PER_ROW))
        past = [p + n for p, n in zip(past, new)]


OUTPUTS = ("r", "p", "g", "beta", "x", "o", "y")


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in OUTPUTS) and torch.equal(a["b"].codes, b["b"].codes)


def same_state(a, b):
    return torch.equal(a.conv, b.conv) and torch.equal(a.delta, b.delta)


@pytest.mark.parametrize("hint,news", [(1, [[1, 1, 1, 1]] * 4), (0, [[3, 1, 40, 2], [40, 2, 1, 3], [46, 0, 0, 0], [0, 20, 0, 20]])])
def test_captured_step_follows_slots_lengths_and_inputs(hint, news):
    a = Layer(4, seed=3)
    a.state.conv.zero_(), a.state.delta.zero_()
    T = sum(news[0])
    h, residual = (torch.zeros(T, a.hidden, dtype=BF16, device=DEV) for _ in range(2))
    kv_len, cu = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(5, dtype=torch.int32, device=DEV)
    for _ in range(2):
        a.step(h, residual, kv_len, cu, hint)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = a.step(h, residual, kv_len, cu, hint)
    past = [0, 7, 0, 2]
    for i, new in enumerate(news):
        if i == 2:
            a.state.slots.copy_(a.state.slots.flip(0))
        b = batch(a, new, past, behind=T - sum(new))
        h.copy_(rand(T, a.hidden, seed=50 + i)), residual.copy_(rand(T, a.hidden, seed=60 + i))
        kv_len.copy_(b.kv_len), cu.copy_(b.cu_q)
        before = a.copy_state()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        after = a.copy_state()
        eager_state = nv().GDNState(before.slots, before.conv.clone(), before.delta.clone())
        want = a.step(h, residual, kv_len, cu, hint, state=eager_state)
        torch.cuda.synchronize()
        assert same(got, want) and same_state(after, eager_state), f"replay {i}"
        a.check(b, before, want)
        past = [p + n for p, n in zip(past, new)]


def delta_call(b, seed, Hk=2, Hv=4, D=128):
    _, q, k, v, g, beta, state = delta_inputs(b, Hk, Hv, D, D, seed)
    args = [x.to(DEV) for x in (q, k, v, g, beta)]
    return args, state.to(DEV), b.slots.to(DEV), b.gpu()


def test_two_captured_graphs_share_a_workspace():
    bs = Seqs([100, 1, 30], [0, 3, 9], seed=1), Seqs([20, 190], [5, 0], seed=2)
    calls = [delta_call(b, 70 + i) for i, b in enumerate(bs)]
    need = [nv().lib.nvfp4_gated_delta_rule_workspace_size(b.T, 0, len(b.new), 2, 4, 128, 128) for b in bs]
    ws = torch.empty(max(need), dtype=torch.uint8, device=DEV)

    def run(i, state, out):
        args, _, slots, lens = calls[i]
        return nv().gated_delta_rule(nv().GDNState(slots, delta=state), *args, *lens, out=out, workspace=ws)

    pools = [c[1].clone() for c in calls]
    outs = [torch.zeros(b.T, 4, 128, dtype=BF16, device=DEV) for b in bs]
    want = []
    for i in range(2):
        s = calls[i][1].clone()
        want.append((run(i, s, torch.zeros_like(outs[i])), s))
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in bs]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            run(i, pools[i], outs[i])
    for order in ((0, 1), (1, 0), (0, 1, 0)):
        ws.random_(0, 256)                       # what it held is of no use to anyone
        for i in order:
            pools[i].copy_(calls[i][1])
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i][0]) and torch.equal(pools[i], want[i][1])


def test_side_streams_at_the_same_time():
    layers = [Layer(3, seed=s) for s in (5, 6)]
    b = batch(layers[0], [70, 1, 5], [0, 0, 0])
    lens = b.gpu()
    hs = [[rand(b.T, 256, seed=80 + 2 * i + j).to(DEV) for j in range(2)] for i in range(2)]
    want, states = [], []
    for a, h in zip(layers, hs):
        s = a.copy_state()
        want.append(a.step(*h, *lens, state=s))
        states.append(s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        got, mine = [None, None], [a.copy_state() for a in layers]
        torch.cuda.synchronize()
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = layers[i].step(*hs[i], *lens, state=mine[i])
        torch.cuda.synchronize()
        for i in range(2):
            used = layers[i].state.slots.long()
            assert same(got[i], want[i])
            assert torch.equal(mine[i].conv[used], states[i].conv[used]) and torch.equal(mine[i].delta[used], states[i].delta[used])


def test_offsets_past_32_bits():
    # rows, heads and slots more than 2^32 bytes apart give what packed ones give
    far = torch.empty((1 << 32) + (1 << 28), dtype=BF16, device=DEV)
    n = 130
    pitch = (1 << 25) - 64
    x, z = rand(n, 4, 64, seed=90).to(DEV), rand(n, 4, 64, seed=91).to(DEV)
    w = rand(64, seed=92, dtype=F32).to(DEV)
    xv = far.as_strided((n, 4, 64), (pitch, 128, 1))
    zv = far.as_strided((n, 4, 64), (pitch, 128, 1), 1024)
    xv.copy_(x), zv.copy_(z)
    out = far.as_strided((n, 256), (pitch, 1), 2048)
    y, _ = nv().gated_rms_norm(xv, zv, w, out=out)
    assert y.data_ptr() == out.data_ptr() and torch.equal(out, nv().gated_rms_norm(x, z, w)[0])
    flat, wide = x.flatten(1), rand(256, seed=93, dtype=F32).to(DEV)
    rows = far.as_strided((n, 256), (pitch, 1), 4096)
    rows.copy_(flat)
    y, _, r = nv().add_rms_norm(rows, wide, rows, out=out, residual_out=rows)
    want, _, want_r = nv().add_rms_norm(flat, wide, flat)
    assert torch.equal(out, want) and torch.equal(rows, want_r)

    b = Seqs([n - 1, 1], [0, 4], seed=3)
    lens, slots = b.gpu(), torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    rows.copy_(flat)
    wc = rand(256, 4, seed=94, dtype=F32).to(DEV)
    pool = far.as_strided((2, 3, 256), (1 << 32, 256, 1), 8192)
    near = rand(2, 3, 256, seed=95).to(DEV)
    pool.copy_(near)
    nv().gdn_conv(nv().GDNState(slots, conv=pool), rows, wc, *lens, out=out)
    assert torch.equal(out, nv().gdn_conv(nv().GDNState(slots, conv=near), flat, wc, *lens)) and torch.equal(pool, near)

    _, q, k, v, g, beta, _ = delta_inputs(b, 1, 2, 64, 64, 96)
    q, k, v, g, beta = (t.to(DEV) for t in (q, k, v, g, beta))
    qv = far.as_strided((n, 1, 64), (pitch, 64, 1), 16384)
    kv = far.as_strided((n, 1, 64), (pitch, 64, 1), 16384 + 64)
    tok, head = (1 << 24) - 64, (1 << 31) + (1 << 25)       # token strides of values and outputs are bounded
    vv = far.as_strided((n, 2, 64), (tok, head, 1), 32768)
    ov = far.as_strided((n, 2, 64), (tok, head, 1), 32768 + 64)
    qv.copy_(q), kv.copy_(k), vv.copy_(v)
    pool = torch.empty((1 << 31) + (1 << 16), device=DEV).as_strided((2, 2, 64, 64), (1 << 31, 4096, 64, 1))
    near = rand(2, 2, 64, 64, seed=97, dtype=F32).to(DEV)
    pool.copy_(near)
    for max_q in (0, 1):                         # in blocks, then token by token
        nv().gated_delta_rule(nv().GDNState(slots, delta=pool), qv, kv, vv, g, beta, *lens, max_q=max_q, out=ov)
        want = nv().gated_delta_rule(nv().GDNState(slots, delta=near), q, k, v, g, beta, *lens, max_q=max_q)
        assert torch.equal(ov, want) and torch.equal(pool, near)

"""The paged-cache operators together, as a server runs them: prompts in chunks and single tokens step by step,
captured steps replayed while lengths, pages and inputs change, other streams, the projections' outputs used in
place."""
import pytest
import torch

from tests.gpu_helpers import DEV, nv
from tests.paged_helpers import Batch, assert_close, norm_rope, rope_table, stored

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class Layer:
    """One attention layer's cache and parameters for S sequences, and its steps through the library."""

    def __init__(self, S, Hq, Hk, D, fp8, page, capacity, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.S, self.Hq, self.Hk, self.D, self.g = S, Hq, Hk, D, g
        width = -(-capacity // page)
        P = S * width
        dt = torch.uint8 if fp8 else BF16
        self.table = torch.randperm(P, generator=g).view(S, width).to(torch.int32)
        k = torch.zeros(P, Hk, page, D, dtype=dt, device=DEV)
        s = torch.full((1,), 5.0 / 448, device=DEV) if fp8 else None
        self.kv = nv().PagedKV(k, torch.zeros_like(k), self.table.to(DEV), s, s)
        self.qw, self.kw = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
        self.rope = rope_table(capacity, D)
        self.dev = [x.to(DEV) for x in (self.qw, self.kw, self.rope)]
        self.len = [0] * S

    def inputs(self, new):
        return (torch.randn(sum(new), (self.Hq + 2 * self.Hk) * self.D, generator=self.g) * 1.2).to(BF16)

    def parts(self, qkv):
        q, k, v = qkv.split([self.Hq * self.D, self.Hk * self.D, self.Hk * self.D], 1)
        return q.unflatten(1, (-1, self.D)), k.unflatten(1, (-1, self.D)), v.unflatten(1, (-1, self.D))

    def step(self, qkv, kv_len, cu, max_q=0, **out):
        q, k, v = self.parts(qkv)
        qw, kw, rope = self.dev
        q = nv().kv_append(self.kv, k, v, kv_len, cu, k_weight=kw, rope=rope, q=q, q_weight=qw, q_out=out.get("q_out"))
        return q, nv().paged_attention(q, self.kv, kv_len, cu, max_q=max_q, out=out.get("out"))

    def check(self, new, q, out):
        """out against the plain attention over the cache as it is."""
        b = Batch.__new__(Batch)
        fp8 = self.kv.k.dtype == torch.uint8
        b.new, b.kv, b.Hq, b.Hk, b.D, b.fp8, b.page = new, self.len, self.Hq, self.Hk, self.D, fp8, self.kv.k.shape[2]
        b.width, b.table, b.k, b.v = self.table.shape[1], self.table, self.kv.k.cpu(), self.kv.v.cpu()
        b.ks = b.vs = self.kv.k_scale.cpu() if fp8 else None
        b.cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        b.T, b.q = sum(new), q.cpu()
        want, _, tol, _ = b.attention()
        assert_close(out, want, tol)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("D,Hq,Hk", [(128, 10, 2), (64, 8, 8), (256, 8, 1)])
def test_prompts_in_chunks_then_single_tokens(fp8, D, Hq, Hk):
    a = Layer(3, Hq, Hk, D, fp8, 16, 400, seed=D)
    first = {}
    for new in ([150, 7, 0], [37, 100, 60], [1, 1, 1], [1, 0, 1], [4, 4, 4], [1, 1, 1]):
        qkv = a.inputs(new)
        before = list(a.len)
        a.len = [x + n for x, n in zip(a.len, new)]
        kv_len = torch.tensor(a.len, dtype=torch.int32, device=DEV)
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
        q, out = a.step(qkv.to(DEV), kv_len, cu, max_q=max(new))
        pos = torch.cat([torch.arange(b, b + n) for b, n in zip(before, new)])
        y, tol = norm_rope(a.parts(qkv)[0], a.qw, a.rope, pos, False)
        assert_close(q, y, stored(y, tol, BF16), "q")
        a.check(new, q, out)
        # earlier tokens' keys stay as they were
        k = a.kv.k[a.kv.page_table.long()].transpose(1, 2).flatten(2, 3).cpu().view(torch.uint8)
        for s in range(3):
            if s in first:
                n, rows = first[s]
                assert torch.equal(k[s, :, :n], rows)
            first[s] = (a.len[s], k[s, :, :a.len[s]].clone())


def test_one_chunk_or_many_give_the_same_cache_and_nearly_the_same_answers():
    outs, caches = [], []
    for chunks in ([300], [130, 170], [299, 1], [100, 3, 197]):
        a = Layer(1, 10, 2, 128, True, 32, 320, seed=5)
        qkv = a.inputs([300]).to(DEV)
        got, at = [], 0
        for n in chunks:
            kv_len = torch.tensor([at + n], dtype=torch.int32, device=DEV)
            cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            got.append(a.step(qkv[at:at + n], kv_len, cu, max_q=n)[1])
            at += n
        outs.append(torch.cat(got).float())
        caches.append(a.kv.k[a.kv.page_table.long()].cpu())
    for o, c in zip(outs[1:], caches[1:]):
        assert torch.equal(c, caches[0])
        # both within 2^-8 |o| (bf16 output) and 2^-11 sum p|v| of the exact answer; |v| is below 6
        assert ((o - outs[0]).abs() <= 2.0 ** -7 * outs[0].abs() + 2.0 ** -10 * 6).all()


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 1, 40, 2]])
def test_captured_step_follows_lengths_pages_and_inputs(new):
    a = Layer(4, 10, 2, 128, True, 16, 3000, seed=9)
    T = sum(new)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
    kv_len = torch.zeros(4, dtype=torch.int32, device=DEV)
    qkv = torch.zeros(T, 14 * 128, dtype=BF16, device=DEV)
    q_out, out = (torch.empty(T, 10, 128, dtype=BF16, device=DEV) for _ in range(2))
    lens = [[50, 1000, 40, 2], [2000, 40, 2990, 700], [3, 1, 40, 2], [2999, 2999, 2999, 2999]]
    a.kv.k.random_(0, 120)                       # finite bytes everywhere
    a.kv.v.random_(0, 120)
    kv_len.copy_(torch.tensor(lens[0], dtype=torch.int32))
    for _ in range(2):
        a.step(qkv, kv_len, cu, q_out=q_out, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(qkv, kv_len, cu, q_out=q_out, out=out)
    for i in range(4):
        qkv.copy_(a.inputs(new))
        kv_len.copy_(torch.tensor(lens[i], dtype=torch.int32))
        if i == 2:
            a.table = a.table.flip(1).contiguous()
            a.kv.page_table.copy_(a.table)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), q_out.clone(), a.kv.k.clone()
        q, want = a.step(qkv, kv_len, cu)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], q) and torch.equal(got[2], a.kv.k), f"replay {i}"
        a.len = lens[i]
        a.check(new, q, want)


def test_two_captured_graphs_share_a_workspace():
    a = Layer(2, 10, 2, 128, True, 16, 2048, seed=11)
    a.kv.k.random_(0, 120)
    a.kv.v.random_(0, 120)
    kv_len = torch.tensor([2000, 77], dtype=torch.int32, device=DEV)
    cu1, cu2 = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1, 2], [0, 60, 61]))
    q1, q2 = (torch.randn(n, 10, 128, device=DEV).to(BF16) for n in (2, 61))
    need = max(nv().lib.nvfp4_paged_attention_workspace_size(n, 0, 2, 10, 2, 128, 2) for n in (2, 61))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
    run1 = lambda o: nv().paged_attention(q1, a.kv, kv_len, cu1, out=o, workspace=ws)  # noqa: E731
    run2 = lambda o: nv().paged_attention(q2, a.kv, kv_len, cu2, out=o, workspace=ws)  # noqa: E731
    run1(o1), run2(o2)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        run1(o1)
    with torch.cuda.graph(g2):
        run2(o2)
    want1, want2 = run1(torch.empty_like(o1)).clone(), run2(torch.empty_like(o2)).clone()
    for _ in range(3):
        o1.zero_(), o2.zero_()
        g1.replay(), g2.replay(), g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want1) and torch.equal(o2, want2)


def test_side_streams_at_the_same_time():
    layers = [Layer(2, 10, 2, 128, True, 16, 1024, seed=s) for s in (1, 2)]
    cu = torch.tensor([0, 1, 40], dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([900, 500], dtype=torch.int32, device=DEV)
    qkvs = [a.inputs([1, 39]).to(DEV) for a in layers]
    for a in layers:
        a.kv.k.random_(0, 120)
        a.kv.v.random_(0, 120)
    want = [a.step(x, kv_len, cu)[1].clone() for a, x in zip(layers, qkvs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = layers[i].step(qkvs[i], kv_len, cu)[1]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_attention_output_feeds_the_quantized_output_projection():
    # append, attention, and the o projection of the framework on the heads' output, in one stream of calls
    a = Layer(2, 8, 2, 128, True, 16, 64, seed=3)
    new = [20, 1]
    a.len = [20, 1]
    kv_len = torch.tensor(a.len, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 20, 21], dtype=torch.int32, device=DEV)
    q, out = a.step(a.inputs(new).to(DEV), kv_len, cu)
    a.check(new, q, out)
    w = nv().quantize(torch.randn(256, 1024, device=DEV).to(BF16))
    y = nv().gemm(nv().quantize(out.flatten(1), "per_row"), w, torch.float32)
    again = nv().gemm(nv().quantize(out.flatten(1).clone(), "per_row"), w, torch.float32)
    assert y.shape == (21, 256) and torch.isfinite(y).all() and torch.equal(y, again)

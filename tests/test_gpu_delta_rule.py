"""The gated delta rule against the 64-bit recurrence: single tokens, drafts, chunks and prompts, head layouts and sizes,
strides, strong and no decays, rows of nobody, slots that are none, values that are not finite."""
import pytest
import torch

from tests.gdn_helpers import BF16, F32, Seqs, assert_within, delta_inputs, delta_rule, rand
from tests.gpu_helpers import DEV, nv

pytestmark = pytest.mark.gpu


def run(b, q, k, v, g, beta, state, max_q=0, scale=None, slots=True):
    """The library's (out with NaN where it writes nothing, states)."""
    st = nv().GDNState(b.slots.to(DEV) if slots else None, delta=state.to(DEV))
    out = torch.full((b.T,) + v.shape[1:], float("nan"), dtype=BF16, device=DEV)
    got = nv().gated_delta_rule(st, q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), *b.gpu(), scale=scale, max_q=max_q, out=out)
    assert got.data_ptr() == out.data_ptr()
    return out, st.delta


def check(b, Hk, Hv, Dk, Dv, max_q=0, seed=0, strong=False, scale=None):
    _, q, k, v, g, beta, state = delta_inputs(b, Hk, Hv, Dk, Dv, seed, strong)
    out, states = run(b, q, k, v, g, beta, state, max_q, scale)
    o, o_tol, s, s_tol = delta_rule(b, q, k, v, g, beta, state, scale)
    assert_within(out, o, o_tol, "out")
    assert_within(states, s, s_tol, "states")


LENGTHS = [([1], [0]), ([1], [5]), ([1, 1, 1], [3, 0, 1]), ([4, 0, 2, 7], [9, 9, 0, 1]), ([15, 16, 17, 18], [0, 3, 0, 3]),
           ([63], [2]), ([64], [0]), ([65], [2]), ([127, 1, 128], [0, 4, 4]), ([129, 200, 1, 0, 33], [0, 1, 1, 5, 0]), ([300], [0])]


@pytest.mark.parametrize("new,past", LENGTHS)
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(2, 4, 128, 128), (1, 3, 64, 64)])
@pytest.mark.parametrize("hint", ["none", "true", "small"])
def test_lengths(new, past, Hk, Hv, Dk, Dv, hint):
    check(Seqs(new, past, front=1, behind=2), Hk, Hv, Dk, Dv, max_q={"none": 0, "true": max(new), "small": 1}[hint])


def test_a_hint_far_past_the_batch():
    check(Seqs([70, 3], [0, 2]), 1, 2, 64, 64, max_q=2 ** 63 - 1)


@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 128, 32), (1, 1, 64, 512), (3, 3, 128, 96), (2, 10, 128, 160), (16, 32, 128, 128), (16, 48, 64, 64)])
def test_heads_and_sizes(Hk, Hv, Dk, Dv):
    check(Seqs([70, 1, 5], [3, 2, 0]), Hk, Hv, Dk, Dv, seed=3)


@pytest.mark.parametrize("Hk,Hv,Dk,Dv,new", [(2, 40, 128, 128, [300, 130, 1]), (40, 40, 64, 128, [65, 20, 400]), (3, 9, 128, 512, [129, 448]),
                                             (1, 33, 64, 160, [1000])])
def test_many_columns(Hk, Hv, Dk, Dv, new):
    # more slices of 16 columns than compute units: the scan takes 32 at a time
    check(Seqs(new, [5] * len(new)), Hk, Hv, Dk, Dv, max_q=max(new), seed=4)


@pytest.mark.parametrize("new", [[5, 3], [150, 80]])
def test_strong_decays_and_scale(new):
    check(Seqs(new, [4, 0]), 2, 4, 128, 64, seed=5, strong=True, scale=1.0)


@pytest.mark.parametrize("n", [3, 100])
@pytest.mark.parametrize("case", ["resets", "none", "beta0", "beta1", "beta2", "zero keys", "same keys", "tiny", "huge"])
def test_corners(n, case):
    b = Seqs([n, n], [7, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=9)
    q, k, v = q.clone(), k.clone(), v.clone()
    if case == "resets":
        g[::3], g[1::7] = -1e4, -float("inf")
    elif case == "none":
        g[:] = 0.0
    elif case.startswith("beta"):
        beta[:] = float(case[-1])
    elif case == "zero keys":
        k[::2], q[1::3] = 0.0, 0.0
    elif case == "same keys":
        k[:] = k[:1]
        beta[:], g[:] = 1.0, 0.0
    else:
        f = 1e-30 if case == "tiny" else 1e30
        v, state = (v.float() * f).to(BF16), state * f
        k, q = (k.float() * (1e-10 if case == "tiny" else 1e10)).to(BF16), (q.float() * 1e12).to(BF16)
        if case == "tiny":
            k[1::2] = (k[1::2].float() * 1e12).to(BF16)
    out, states = run(b, q, k, v, g, beta, state)
    o, o_tol, s, s_tol = delta_rule(b, q, k, v, g, beta, state)
    assert_within(out, o, o_tol + 2.0 ** -133, "out")             # bf16's smallest step
    assert_within(states, s, s_tol + 2.0 ** -140, "states")


@pytest.mark.parametrize("n,at", [(4, 1), (200, 70), (200, 63), (200, 0)])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_touch_nothing_before_them(n, at, what, value):
    b = Seqs([n, n], [0, 3])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=11)
    clean = run(b, q, k, v, g, beta, state)
    x = {"q": q, "k": k, "v": v, "g": g, "beta": beta}
    x = {name: t.clone() for name, t in x.items()}
    x[what][(at, 1, 5) if x[what].dim() == 3 else (at, 1)] = value
    out, states = run(b, x["q"], x["k"], x["v"], x["g"], x["beta"], state)
    heads = {"v": [1], "q": [2, 3], "k": [2, 3], "g": [1], "beta": [1]}[what]          # two value heads to a key head
    other = [h for h in range(4) if h not in heads]
    o, o_tol, s, s_tol = delta_rule(b, q, k, v, g, beta, state)
    assert torch.equal(out[:, other], clean[0][:, other]) and torch.equal(out[n:], clean[0][n:])
    assert torch.equal(states[b.slots.long()][:, other], clean[1][b.slots.long()][:, other])
    assert_within(out[:at], o[:at], o_tol[:at], "tokens before")
    if what == "v":
        cols = [c for c in range(64) if c != 5]
        assert not torch.isfinite(out[at:n, 1, 5].float()).any() and not torch.isfinite(states[int(b.slots[0]), 1, :, 5]).all()
        assert_within(out[:n, 1, cols], o[:n, 1, cols], o_tol[:n, 1, cols], "other columns")
        assert_within(states[int(b.slots[0]), 1][:, cols], s[int(b.slots[0]), 1][:, cols], s_tol[int(b.slots[0]), 1][:, cols])
    elif what == "q":
        later = [t for t in range(n) if t != at]
        assert_within(out[later], o[later], o_tol[later], "other tokens")
        assert_within(states, s, s_tol)
    elif not (what == "g" and value > 0):
        assert not torch.isfinite(out[at:n, heads].float()).any() and not torch.isfinite(states[int(b.slots[0]), heads]).all()


def test_strided_operands_and_layouts():
    b = Seqs([90, 3], [1, 0])
    x, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 128, seed=13)
    want, states = run(b, q, k, v, g, beta, state)
    xg = x.to(DEV)
    qs, ks, vs = (xg[:, :256].unflatten(1, (2, 128)), xg[:, 256:512].unflatten(1, (2, 128)), xg[:, 512:].unflatten(1, (4, 128)))
    pool = torch.zeros((b.num_slots, 2, 4, 128, 128), device=DEV)          # one half of a wider pool
    pool[:, 1] = state.to(DEV)
    out = torch.empty((4, b.T, 128), dtype=BF16, device=DEV).transpose(0, 1)
    got = nv().gated_delta_rule(nv().GDNState(b.slots.to(DEV), delta=pool[:, 1]), qs, ks, vs, g.to(DEV), beta.to(DEV), *b.gpu(), out=out)
    assert torch.equal(got, want) and torch.equal(pool[:, 1], states) and (pool[:, 0] == 0).all()


def test_slots_that_are_none_and_no_slots():
    b = Seqs([70, 1, 2, 66], [5, 5, 5, 5])
    b.slots[1], b.slots[3] = -1, b.num_slots
    check(b, 1, 2, 128, 64, seed=15)
    b = Seqs([70, 1, 2], [5, 0, 5])
    b.slots = torch.arange(3, dtype=torch.int32)
    _, q, k, v, g, beta, state = delta_inputs(b, 1, 2, 128, 64, seed=16)
    out, states = run(b, q, k, v, g, beta, state, slots=False)
    o, o_tol, s, s_tol = delta_rule(b, q, k, v, g, beta, state)
    assert_within(out, o, o_tol)
    assert_within(states, s, s_tol)


def test_pieces_of_a_sequence_go_on_from_each_other():
    n, cuts = 260, [0, 1, 65, 66, 70, 230, 260]
    b = Seqs([n], [0], spare=0)
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=17)
    o, o_tol, s, s_tol = delta_rule(b, q, k, v, g, beta, state)
    st = nv().GDNState(None, delta=torch.full(state.shape, float("nan"), device=DEV))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    outs = [nv().gated_delta_rule(st, *(x[a:z].to(DEV) for x in (q, k, v, g, beta)), i32(z), i32(0, z - a)) for a, z in zip(cuts, cuts[1:])]
    assert_within(torch.cat(outs), o, o_tol)
    assert_within(st.delta, s, s_tol)


def test_same_bits_every_time():
    b = Seqs([190, 1, 64], [1, 1, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 128, seed=19)
    first = run(b, q, k, v, g, beta, state)
    for _ in range(3):
        again = run(b, q, k, v, g, beta, state)
        assert torch.equal(first[0][b.rows().to(DEV)], again[0][b.rows().to(DEV)]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("max_q", [0, 1])
def test_lengths_out_of_range_stay_inside(max_q):
    b = Seqs([8], [0], spare=0)
    _, q, k, v, g, beta, state = delta_inputs(b, 1, 2, 64, 32, seed=21)
    for cu in ([-5, 3, 100], [4, 2, 6], [2 ** 31 - 1, 0, 8], [-2 ** 31, 2 ** 31 - 1, 0]):
        pool, guard = torch.zeros((6, 2, 64, 32), device=DEV), torch.full((24, 2, 32), 3.0, dtype=BF16, device=DEV)
        st = nv().GDNState(torch.tensor([0, 1], dtype=torch.int32, device=DEV), delta=pool[2:4])
        nv().gated_delta_rule(st, *(x.to(DEV) for x in (q, k, v, g, beta)), torch.tensor([9, 2 ** 31 - 1], dtype=torch.int32, device=DEV),
                              torch.tensor(cu, dtype=torch.int32, device=DEV), max_q=max_q, out=guard[8:16])
        assert (guard[:8] == 3).all() and (guard[16:] == 3).all() and (pool[:2] == 0).all() and (pool[4:] == 0).all()

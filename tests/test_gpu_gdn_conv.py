"""The causal convolution with its states against the 64-bit formula: widths, types, sequences of any length in any
order, runs that cross sequences, states moved by fewer tokens than they hold, rows of nobody, slots that are none."""
import pytest
import torch

from tests.gdn_helpers import BF16, F32, HALF, Seqs, assert_within, conv, rand
from tests.gpu_helpers import DEV, nv

pytestmark = pytest.mark.gpu


def check(b, C, W, dtype=BF16, out_dtype=BF16, bias=True, seed=0, slots=True):
    x, w = rand(b.T, C, seed=seed, dtype=dtype, scale=1.5), rand(C, W, seed=seed + 1, dtype=F32, scale=0.6)
    bb = rand(C, seed=seed + 2, dtype=F32, scale=0.2) if bias else None
    state = rand(b.num_slots, W - 1, C, seed=seed + 3, dtype=dtype)
    if not slots:
        b.slots = torch.arange(len(b.new), dtype=torch.int32)
    y, tol, want = conv(b, x, w, bb, state)
    wide = torch.full((b.T, C + 40), float("nan"), dtype=dtype, device=DEV)
    wide[:, 8:C + 8] = x.to(DEV)
    st = nv().GDNState(b.slots.to(DEV) if slots else None, conv=state.to(DEV))
    out = torch.full((b.T, C), float("nan"), dtype=out_dtype, device=DEV)
    got = nv().gdn_conv(st, wide[:, 8:C + 8], w.to(DEV), *b.gpu(), bias=None if bb is None else bb.to(DEV), out_dtype=out_dtype, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert_within(got, y, tol + HALF[out_dtype] * y.abs())       # rows of nobody: still NaN
    assert torch.equal(st.conv.cpu(), want)
    return got, st


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [9]), ([1, 2, 3, 4, 5], [7, 1, 0, 3, 9]), ([0, 2, 0, 0, 1, 3], [4, 4, 0, 4, 0, 4]),
                                      ([100], [3]), ([17, 1, 1, 40, 3], [0, 2, 0, 5, 9])])
def test_sequences(W, dtype, out_dtype, new, past):
    check(Seqs(new, past, front=2, behind=3), 72, W, dtype, out_dtype, bias=W != 3)


@pytest.mark.parametrize("C", [8, 504, 512, 520, 1032, 8192])
def test_channels(C):
    check(Seqs([3, 5, 1], [2, 0, 8]), C, 4)


@pytest.mark.parametrize("seed", range(4))
def test_long_runs_cross_sequences_of_every_length(seed):
    # enough tokens and channels that a wavefront takes 16 tokens at a time
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(0, [3, 8, 30, 700][seed], ([6000, 2500, 600, 24][seed],), generator=g).tolist()
    past = [int(p) for p in torch.randint(0, 3, (len(new),), generator=g)]
    b = Seqs(new, past, front=5, behind=21, seed=seed)
    x, w = rand(b.T, 8192, seed=seed), rand(8192, 4, seed=seed + 1, dtype=F32, scale=0.6)
    state = rand(b.num_slots, 3, 8192, seed=seed + 3)
    st = nv().GDNState(b.slots.to(DEV), conv=state.to(DEV))
    out = torch.full((b.T, 8192), float("nan"), dtype=BF16, device=DEV)
    nv().gdn_conv(st, x.to(DEV), w.to(DEV), *b.gpu(), out=out)
    some = torch.tensor([0, 7, 511, 512, 4099, 8191])
    y, tol, want = conv(b, x[:, some], w[some], None, state[:, :, some])
    assert_within(out[:, some.to(DEV)], y, tol + HALF[BF16] * y.abs())
    assert torch.equal(st.conv.cpu()[:, :, some], want)


def test_slots_that_are_none_and_no_slots():
    b = Seqs([4, 1, 2, 6], [5, 5, 5, 5])
    b.slots[1], b.slots[3] = -1, b.num_slots
    check(b, 64, 4)
    check(Seqs([4, 1, 2], [5, 0, 5]), 64, 4, slots=False)


def test_one_token_at_a_time_gives_the_same_bits():
    C, n = 96, 9
    x, w = rand(n, C, seed=1).to(DEV), rand(C, 4, seed=2, dtype=F32).to(DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    whole = nv().GDNState(None, conv=torch.zeros((1, 3, C), dtype=BF16, device=DEV))
    y = nv().gdn_conv(whole, x, w, i32(n), i32(0, n))
    step = nv().GDNState(None, conv=torch.full((1, 3, C), float("nan"), dtype=BF16, device=DEV))
    for t in range(n):
        assert torch.equal(nv().gdn_conv(step, x[t:t + 1], w, i32(t + 1), i32(0, 1))[0], y[t])
    assert torch.equal(step.conv, whole.conv)


def test_nan_stays_in_its_sequence_channel_and_window():
    b = Seqs([6, 6], [0, 0])
    x, w = rand(12, 64, seed=3), rand(64, 4, seed=4, dtype=F32)
    x[1, 10], x[8, 20] = float("nan"), float("inf")
    st = nv().GDNState(None, conv=torch.zeros((2, 3, 64), dtype=BF16, device=DEV))
    got = nv().gdn_conv(st, x.to(DEV), w.to(DEV), *b.gpu()).cpu()
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[1:5, 10] = True
    assert torch.equal(bad[:, :20], want[:, :20]) and not bad[:8, 20].any() and not bad[:, 21:].any()


def test_lengths_out_of_range_stay_inside():
    # cu_q out of order or range: some rows are computed, none outside the tensors is touched
    x, w = rand(8, 64, seed=5).to(DEV), rand(64, 4, seed=6, dtype=F32).to(DEV)
    for cu in ([-5, 3, 100], [4, 2, 6], [2 ** 31 - 1, 0, 8], [-2 ** 31, 2 ** 31 - 1, 0]):
        pool = torch.zeros((6, 3, 64), dtype=BF16, device=DEV)
        guard = torch.full((24, 64), 3.0, dtype=BF16, device=DEV)
        st = nv().GDNState(torch.tensor([0, 1], dtype=torch.int32, device=DEV), conv=pool[2:4])
        nv().gdn_conv(st, x, w, torch.tensor([9, 2 ** 31 - 1], dtype=torch.int32, device=DEV),
                      torch.tensor(cu, dtype=torch.int32, device=DEV), out=guard[8:16])
        assert (guard[:8] == 3).all() and (guard[16:] == 3).all() and (pool[:2] == 0).all() and (pool[4:] == 0).all()

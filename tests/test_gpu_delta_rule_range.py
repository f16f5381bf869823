"""Values of one block that lie far apart: a token has no influence on those before it, however large it is, and what
follows a reset is exact, however large the state was."""
import pytest
import torch

from tests.delta_range_helpers import exact_rule
from tests.gdn_helpers import Seqs, assert_within, delta_inputs
from tests.test_gpu_delta_rule import run

pytestmark = pytest.mark.gpu

SIZES = [8, 16, 22, 30, 40, 60, 88]


def check(b, q, k, v, g, beta, state):
    out, states = run(b, q, k, v, g, beta, state)
    o, o_tol, s, s_tol = exact_rule(b, q, k, v, g, beta, state)
    assert_within(out, o, o_tol, "out")
    assert_within(states, s, s_tol, "states")
    return out


@pytest.mark.parametrize("n,at", [(16, 9), (17, 9), (100, 50), (100, 70), (200, 63), (200, 128)])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("columns", ["all", "one"])
def test_a_large_token(n, at, size, columns):
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=35)
    v = v.float()
    rows = [at, n + at]
    if columns == "all":
        v[rows] *= 2.0 ** size
    else:
        v[rows, 1, 5] *= 2.0 ** size
    check(b, q, k, v.bfloat16(), g, beta, state)


@pytest.mark.parametrize("n,at", [(16, 9), (17, 9), (100, 50), (100, 70), (200, 63), (200, 128)])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("decay", ["reset", "steep"])
def test_a_large_state_that_is_forgotten(n, at, size, decay):
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=37)
    state = state * 2.0 ** size
    if decay == "reset":
        g[[at, n + at]] = -1e4
    else:
        g[at:at + 6], g[n + at:n + at + 6] = -0.12 * size, -0.12 * size          # e^-0.72 size = 2^-1.04 size
    check(b, q, k, v, g, beta, state)


@pytest.mark.parametrize("n", [60, 100, 260])
@pytest.mark.parametrize("strong", [False, True])
def test_tokens_of_zeros(n, strong):
    # padding in front, within and behind: rows of zeros write nothing, whatever decays
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=39, strong=strong)
    q, k, v = q.clone(), k.clone(), v.clone()
    for lo, hi in ((0, 20), (30, 33), (40, 45), (n - 10, n), (n, n + 25)):
        q[lo:hi], k[lo:hi], v[lo:hi] = 0.0, 0.0, 0.0
    out = check(b, q, k, v, g, beta, state)
    assert (out[:20] == 0).all() and (out[n:n + 25] == 0).all()


@pytest.mark.parametrize("n", [17, 100])
@pytest.mark.parametrize("size", [16, 24, 40])
def test_strengths_near_none(n, size):
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=41)
    beta[::3] = 2.0 ** -size
    check(b, q, k, v, g, beta, state)


@pytest.mark.parametrize("n", [100, 200])
def test_closed_gates_beside_weak_decays_stay_in_blocks(n):
    # strengths of 1e-9 behind the first token: nothing is lost, what was written before is still there.  That the blocks keep
    # them shows in the states' last bits, which differ from the token-by-token kernel's
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=47)
    g[:] = -2.0 ** -7
    beta[1::2] = 1e-9
    check(b, q, k, v, g, beta, state)
    blocks, steps = (run(b, q, k, v, g, beta, state, max_q=m)[1][b.slots.long()] for m in (0, 1))
    assert (blocks != steps).flatten(2).any(2).all()


@pytest.mark.parametrize("n", [100, 200])
def test_slices_out_of_range_are_the_step_kernels(n):
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=49)
    v = v.clone()
    v[[40, n + 40], :, 32:] *= 2.0 ** 60
    blocks, steps = (run(b, q, k, v, g, beta, state, max_q=m)[1][b.slots.long()] for m in (0, 1))
    assert torch.equal(blocks[..., 32:], steps[..., 32:])
    assert (blocks != steps)[..., :32].flatten(2).any(2).all()


@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(2, 40, 128, 128), (3, 72, 64, 64), (1, 2, 64, 32)])
@pytest.mark.parametrize("case", ["large token", "large column", "forgotten", "padding", "first columns zero", "large behind zeros", "reset"])
def test_wide_slices_and_short_keys(Hk, Hv, Dk, Dv, case):
    # more slices of 16 columns than compute units are taken 32 at a time
    n = 150
    b = Seqs([n, 40], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, Hk, Hv, Dk, Dv, seed=53)
    q, k, v = q.clone(), k.clone(), v.clone()
    if case == "large token":
        v[[50, n + 20]] *= 2.0 ** 40
    elif case == "large column":
        v[[50, n + 20], :, 21] *= 2.0 ** 40
    elif case == "forgotten":
        state, g[[70, n + 9]] = state * 2.0 ** 40, -1e4
    elif case == "padding":
        for x in (q, k, v):
            x[20:30], x[64:140], x[n:n + 5] = 0.0, 0.0, 0.0
    elif case == "first columns zero":
        v[::2, :, :4], v[1::2, :, 16:20] = 0.0, 0.0
    elif case == "large behind zeros":         # the first four columns tell nothing of the large token's row
        v[:, :, :5], v[:, :, 16:21] = 0.0, 0.0
        v[[50, n + 20]] *= 2.0 ** 40
    else:
        state, g[[70, n + 9]], beta[64:] = state * 2.0 ** 60, -1e4, 0.0
    check(b, q, k, v, g, beta, state)


@pytest.mark.parametrize("n", [9, 100])
@pytest.mark.parametrize("size", [40, 80, 100, 110, 116])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(2, 4, 128, 64), (2, 40, 128, 128)])
def test_small_values_are_large_ones_scaled(n, size, Hk, Hv, Dk, Dv):
    # the rule is linear in v and the state, and a power of two changes no bits but where numbers end: two outputs are apart by
    # the two roundings to bf16 (2^-8 each), 32-bit arithmetic (2^-15 of the largest) and bf16's smallest step, states by that alone
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, Hk, Hv, Dk, Dv, seed=55)
    out, states = (x.double().cpu() for x in run(b, q, k, v, g, beta, state))
    small, small_states = (x.double().cpu() for x in run(b, q, k, (v.float() * 2.0 ** -size).bfloat16(), g, beta, state * 2.0 ** -size))
    f = 2.0 ** -size
    assert_within(small, out * f, 2.0 ** -7 * out.abs() * f + 2.0 ** -15 * out.abs().amax() * f + 2.0 ** -133)
    assert_within(small_states, states * f, 2.0 ** -18 * states.abs().amax() * f + 2.0 ** -148)

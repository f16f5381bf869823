"""States of every size that decay to nothing inside a block in which nothing is written."""
import pytest
import torch

from tests.delta_range_helpers import exact_rule
from tests.gdn_helpers import Seqs, assert_within, delta_inputs
from tests.test_gpu_delta_rule import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [9, 17, 65, 200])
@pytest.mark.parametrize("size", [0, 20, 21, 24, 60, 90])
@pytest.mark.parametrize("nothing", ["beta", "v"])
@pytest.mark.parametrize("decay", ["reset", "-inf", "-8", "-1"])
def test_nothing_written_while_the_state_decays(n, size, nothing, decay):
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=31)
    v, state = v.clone(), state * 2.0 ** size
    (beta if nothing == "beta" else v)[:] = 0.0
    if decay in ("reset", "-inf"):
        g[n // 2::n] = -1e4 if decay == "reset" else -float("inf")
    else:
        g[:] = float(decay)
    out, states = run(b, q, k, v, g, beta, state)
    o, o_tol, s, s_tol = exact_rule(b, q, k, v, g, beta, state)
    assert_within(out, o, o_tol, "out")
    assert_within(states, s, s_tol, "states")
    if decay in ("reset", "-inf"):             # exactly nothing behind it
        mine = states[b.slots.long()]
        assert (out[n // 2:n] == 0).all() and (out[n:] == 0).all() and (mine == 0).all()


@pytest.mark.parametrize("nothing", ["beta", "v"])
def test_a_bound_that_grew_over_blocks(nothing):
    # |beta v| of about 1000 and decays near none for 40 blocks, then a reset in a block that writes nothing
    n, at = 40 * 64 + 100, 40 * 64
    b = Seqs([n], [0])
    _, q, k, v, g, beta, state = delta_inputs(b, 1, 2, 128, 32, seed=33)
    v, g = (v.float() * 1000).to(v.dtype), g * 0 - 2.0 ** -12
    g[at + 5] = -1e4
    (beta if nothing == "beta" else v)[at:at + 64] = 0.0
    out, states = run(b, q, k, v, g, beta, state)
    o, o_tol, s, s_tol = exact_rule(b, q, k, v, g, beta, state)
    assert_within(out, o, o_tol + 2.0 ** -26 * o.abs().amax(), "out")      # M grows by 64 |beta v| a block: 2^5 blocks more of it
    assert_within(states, s, s_tol + 2.0 ** -26 * s.abs().amax(), "states")
    assert (out[at + 5:at + 64] == 0).all()


@pytest.mark.parametrize("n", [9, 100, 200])
def test_a_decay_to_zero_is_any_other_reset(n):
    # e^-inf = e^-1e4 = 0: the same bits, and no reason to leave the blocks
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=35)
    g[5::17] = -1e4
    out, states = run(b, q, k, v, g, beta, state)
    g[5::17] = -float("inf")
    again, states_again = run(b, q, k, v, g, beta, state)
    assert torch.equal(out, again) and torch.equal(states, states_again)

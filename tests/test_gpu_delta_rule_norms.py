"""Queries and keys of every length, token by token and in blocks: 1e-6 beside the squares' sum, never beside less."""
import pytest
import torch

from tests.delta_range_helpers import exact_rule
from tests.gdn_helpers import Seqs, assert_within, delta_inputs
from tests.test_gpu_delta_rule import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [3, 100])
@pytest.mark.parametrize("Dk", [64, 128])
@pytest.mark.parametrize("length", [1e-18, 1e-4, 1e-3, 1.0, 1e10, 1e14, 2e15, 1e16, 1e18, 1e21, 1e30, 3e37])
def test_rows_of_every_length(n, Dk, length):
    b = Seqs([n, n], [4, 0])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, Dk, 64, seed=43)
    q, k = ((x.float() * (length / x.float().norm(dim=-1, keepdim=True))).bfloat16() for x in (q, k))
    out, states = run(b, q, k, v, g, beta, state)
    o, o_tol, s, s_tol = exact_rule(b, q, k, v, g, beta, state)
    assert_within(out, o, o_tol, "out")
    assert_within(states, s, s_tol, "states")


def test_a_redone_slice_of_long_rows():
    # a strength past 2 makes the blocks leave the head to the token-by-token kernel
    b = Seqs([100], [4])
    _, q, k, v, g, beta, state = delta_inputs(b, 1, 2, 128, 32, seed=45)
    q, k = ((x.float() * 1e17).bfloat16() for x in (q, k))
    beta[90, 0] = 2.5
    out, states = run(b, q, k, v, g, beta, state)
    o, o_tol, s, s_tol = exact_rule(b, q, k, v, g, beta, state)
    assert_within(out[:90], o[:90], o_tol[:90], "out")
    assert_within(out[:, 1], o[:, 1], o_tol[:, 1], "the other head")

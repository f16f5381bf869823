"""The gated delta rule's outputs within 32-bit arithmetic and their own rounding to bf16, whatever kernel a length goes to."""
import pytest
import torch

from tests.delta_range_helpers import exact_rule
from tests.gdn_helpers import Seqs, assert_within, delta_inputs
from tests.test_gpu_delta_rule import run

pytestmark = pytest.mark.gpu


def check(b, q, k, v, g, beta, state, scale=None):
    out, states = run(b, q, k, v, g, beta, state, scale=scale)
    o, o_tol, s, s_tol = exact_rule(b, q, k, v, g, beta, state, scale)
    assert_within(out, o, o_tol, "out")
    assert_within(states, s, s_tol, "states")
    return out, states


@pytest.mark.parametrize("new,past", [([16], [3]), ([17], [3]), ([64, 130], [0, 5]), ([300, 1], [2, 9]), ([20] * 6, [1] * 6)])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(2, 4, 128, 128), (1, 3, 64, 64), (2, 40, 128, 128), (1, 3, 128, 96)])
@pytest.mark.parametrize("strong", [False, True])
def test_outputs_to_32_bits(new, past, Hk, Hv, Dk, Dv, strong):
    b = Seqs(new, past, front=1, behind=2)
    _, q, k, v, g, beta, state = delta_inputs(b, Hk, Hv, Dk, Dv, seed=23, strong=strong)
    check(b, q, k, v, g, beta, state)


@pytest.mark.parametrize("n", [16, 17, 100])
def test_queries_across_a_dominant_write(n):
    # every key the same, queries nearly orthogonal to it: outputs far below what the state holds
    b = Seqs([n], [4])
    _, q, k, v, g, beta, state = delta_inputs(b, 2, 4, 128, 64, seed=25)
    k, v, state = k.clone(), v.clone(), state * 2.0 ** -12
    k[:] = k[:1]
    a = k[0].double()
    along = (q.double() * a).sum(-1, keepdim=True) / (a * a).sum(-1, keepdim=True)
    q = (q.double() - along * a).to(torch.bfloat16)
    beta[:], g[:] = 1.0, 0.0
    check(b, q, k, v, g, beta, state)

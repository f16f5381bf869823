"""Operands of the Gated DeltaNet operators that the binding takes, without a GPU: past every check but the last, that the
tensors are on a GPU."""
import pytest
import torch

import nvfp4_w4a4_block_amd as nv


@pytest.mark.parametrize("strides", [(1, 1), (1, 7), (1, 0)])
@pytest.mark.parametrize("T", [1, 5])
def test_gates_of_one_value_head_whatever_the_stride_of_its_dimension(T, strides):
    bf, i32 = torch.bfloat16, torch.int32
    q, v = torch.zeros(T, 1, 64, dtype=bf), torch.zeros(T, 1, 32, dtype=bf)
    g = torch.zeros(64).as_strided((T, 1), strides)
    assert g.is_contiguous()
    state = nv.GDNState(delta=torch.zeros(1, 1, 64, 32))
    args = torch.tensor([T], dtype=i32), torch.tensor([0, T], dtype=i32)
    with pytest.raises(ValueError, match="GPU"):
        nv.gated_delta_rule(state, q, q, v, g, g, *args)
    with pytest.raises(ValueError, match="GPU"):
        nv.gated_delta_rule(state, q, q, v, g, torch.zeros(T, 1), *args)
    if T > 1:                                   # tokens apart are another matter
        with pytest.raises(ValueError, match="g:"):
            nv.gated_delta_rule(state, q, q, v, torch.zeros(64).as_strided((T, 1), (2, 1)), g, *args)

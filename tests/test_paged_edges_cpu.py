"""Limits and checks of the paged cache's operators that need no GPU: at the C ABI with fake addresses that are never
dereferenced, and in the binding."""
import pytest
import torch

from tests.test_paged_cpu import attend, batch, cache


@pytest.fixture(scope="module")
def nv():
    import nvfp4_w4a4_block_amd as m
    return m


def test_attention_refuses_tables_past_2_30_tokens(nv):
    # positions, block ends and a block's look-ahead are 32-bit numbers in the kernels
    for page in (16, 1024):
        most = (1 << 30) // page
        for width in (most + 1, ((1 << 31) - 1) // page):
            c = cache(nv, page_size=page, table_width=width, table_stride=width, k_page_stride=1 << 20, v_page_stride=1 << 20)
            assert attend(nv, c) == 2, (page, width)
        c = cache(nv, page_size=page, table_width=most, table_stride=most, k_page_stride=1 << 20, v_page_stride=1 << 20)
        assert attend(nv, c, ws=None) == 3          # the next check, of the workspace, is reached

"""Limits and checks of the paged cache's operators that need no GPU: at the C ABI with fake addresses that are never
dereferenced, and in the binding."""
import os
import subprocess

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


def test_a_plan_stays_in_32_bits_whatever_the_sequences(tmp_path):
    # the blocks that the kernel adds up (as many tiles as each sequence's rows fill, times the key blocks of its
    # length) for offsets in order, all alike, and jumping between nothing and all tokens: wherever a plan is
    # allowed the sum and a workgroup's share stay below 2^31, and ordinary batches are allowed one
    src = tmp_path / "plan.cpp"
    src.write_text(r"""
#include "paged_internal.h"
#include <cstdio>
using i64 = long long;
int main() {
  i64 bad = 0, allowed = 0, refused = 0;
  for (i64 S : {1, 2, 16, 64, 300, 511, 1024}) for (i64 T : {1, 64, 512, 4000}) for (i64 G : {1, 5, 16, 32}) for (i64 bm : {16, 32})
  for (i64 hi : {bm, (i64)INT32_MAX}) for (i64 heads : {1, 8, 128}) for (i64 cap : {4, 256, 8192, 1 << 17, 1 << 23}) {
    const i64 slots = hi == bm ? S : T * G / bm + S;
    if (slots > 1024) continue;
    const bool fits = nvfp4::plan_fits(true, slots, S, T * G, hi, bm, cap, heads, 1024);
    (fits ? allowed : refused)++;
    for (int kind = 0; kind < 3; ++kind) {
      i64 sum = 0;
      for (i64 s = 0; s < S; ++s) {
        auto cu = [&](i64 j) { return kind == 0 ? T * j / S : kind == 1 ? (j > S / 2 ? T : 0) : (j & 1 ? T : 0); };
        const i64 n = cu(s + 1) > cu(s) ? cu(s + 1) - cu(s) : 0, rows = n * G;
        if (rows > 0 && rows <= hi) sum += (rows + bm - 1) / bm * cap;
      }
      if (fits && (sum >= INT32_MAX || (sum * heads + 1023) / 1024 >= INT32_MAX)) bad++;
    }
  }
  // 64 decodes over 131072 keys; 1024 over 32768; the tile kernel's slots
  const bool usual = nvfp4::plan_fits(true, 84, 64, 64 * 5, INT32_MAX, 16, 1024, 8, 1024) &&
                     nvfp4::plan_fits(true, 1024, 1024, 1024 * 5, 16, 16, 256, 8, 1024) &&
                     nvfp4::plan_fits(false, 101, 17, 100 * 128, INT32_MAX, 128, 16384, 8, 512);
  printf("%lld %d\n", bad, usual ? 1 : 0);
  return !(bad == 0 && usual && allowed > 100 && refused > 100);
}
""")
    exe = tmp_path / "plan"
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_w4a4_block_amd", "csrc")
    r = subprocess.run(["/opt/rocm/bin/hipcc", "-O1", "-x", "hip", "--cuda-host-only", "-I", csrc, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_binding_takes_a_workspace_of_the_size_asked_for(nv):
    kv, n, cu, q, _ = batch(nv, S=1100, T=1100)
    size = lambda T, S: nv.lib.nvfp4_paged_attention_workspace_size(T, 0, S, 4, 2, 64, 2)  # noqa: E731
    assert size(1100, 1100) == 0 and size(4, 3) > 0
    with pytest.raises(ValueError, match="GPU"):            # nothing else is wrong
        nv.paged_attention(q, kv, n, cu, workspace=torch.empty(size(1100, 1100), dtype=torch.uint8))
    kv, n, cu, q, _ = batch(nv)
    with pytest.raises(ValueError, match="GPU"):
        nv.paged_attention(q, kv, n, cu, workspace=torch.empty(size(4, 3), dtype=torch.uint8))
    for bad in (torch.empty(0), torch.empty(0, dtype=torch.int32), torch.empty(64, 64, dtype=torch.uint8).T, 5,
                torch.empty(0, dtype=torch.uint8), torch.empty(size(4, 3) - 1, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            nv.paged_attention(q, kv, n, cu, workspace=bad)


@pytest.mark.parametrize("fp8", [True, False])
def test_binding_takes_a_single_head_whatever_its_stride(nv, fp8):
    # [pages, page_size, heads, dim] seen as [pages, heads, page_size, dim]: with one head every page is contiguous
    kv, n, cu, q, k = batch(nv, fp8=fp8, Hk=1)
    one = kv.k.reshape(5, 16, 1, 64).transpose(1, 2)
    assert one.shape == kv.k.shape and one.is_contiguous() and one.stride() != kv.k.stride()
    view = nv.PagedKV(one, one, kv.page_table, kv.k_scale, kv.v_scale)
    with pytest.raises(ValueError, match="GPU"):
        nv.paged_attention(q, view, n, cu)
    with pytest.raises(ValueError, match="GPU"):
        nv.kv_append(view, k, k, n, cu)
    for bad in (one[:, :, ::2], one[..., :32], one.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError, match="contiguous"):
            nv.kv_append(nv.PagedKV(bad, bad, kv.page_table, kv.k_scale, kv.v_scale), k, k, n, cu)


def test_launch_limits_are_found_before_anything_is_enqueued(nv):
    # two kernels serve this call; only the second one's grid passes the limit.  (Without a GPU a launch is an error of
    # its own, status 4.)
    q = nv._Heads(0x10000, 256, 256 * 128, 128)
    c = cache(nv, kv_heads=8, num_seqs=2_000_000, k_page_stride=1 << 20, v_page_stride=1 << 20)
    assert attend(nv, c, T=400_000, q=q, out=q, ws=None, wsb=0) == 2

"""The order of M0 writes and direct-to-LDS copies, on generated gfx950 assembly (no GPU)."""
import os
import subprocess

import pytest

from nvfp4_w4a4_block_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    """Device assembly of every source with direct-to-LDS copies."""
    flags = [f for f in b.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    out = {}
    for name in sorted(os.listdir(b.CSRC)):
        path = os.path.join(b.CSRC, name)
        if not name.endswith(".hip") or "global_load_lds" not in open(path).read():
            continue
        asm = tmp_path_factory.mktemp("asm") / (name + ".s")
        r = subprocess.run([b.hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"), path, "-o", str(asm)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        out[name] = asm.read_text()
    return out


def test_every_copy_has_its_m0_write_and_wait_state(listings):
    assert set(listings) == {"gemm.hip", "gdn_chunk.hip"}
    for name, asm in listings.items():
        assert b.check_m0(asm) > 0, name
        code = [l.strip() for l in asm.splitlines()]
        code = [l for l in code if l and not l.startswith((";", "."))]
        copies = [i for i, l in enumerate(code) if l.startswith("global_load_lds")]
        assert len(copies) == b.check_m0(asm)
        assert all(code[i - 1] == "s_nop 0" and code[i - 2].startswith("s_mov_b32 m0, ") for i in copies), name


def test_check_wants_the_wait_state():
    good = "s_mov_b32 m0, s4\ns_nop 0\nglobal_load_lds_dwordx4 v1, off\n"
    assert b.check_m0(2 * good) == 2
    for bad in (good.replace("s_nop 0\n", ""), good.replace("s_nop 0", "s_add_u32 s1, s2, s3"), good + "global_load_lds_dword v1, off\n",
                good + "s_add_u32 s0, m0, 1\n", good.replace("s4", "0x100"), "s_mov_b32 m0, s4\ns_nop 0\n", "s_nop 0\n"):
        with pytest.raises(RuntimeError):
            b.check_m0(bad)


def test_copies_wait_for_reads_in_every_listing(listings):
    for name, asm in listings.items():
        found = b.check_lds_refills(asm)
        assert found, name
        if name == "gdn_chunk.hip":
            assert len(found) == 4 and not any(found.values()), found


def test_loads_and_stores_that_the_ring_counts_on_are_there(listings):
    marks = b.check_ring_marks(listings["gdn_chunk.hip"])
    # two in front of the loop's three copies of the block, two around the first wait, one behind
    assert len(marks) == 4 and all("chunk_scan_kernel" in k and n >= 5 for k, n in marks.items()), marks
    assert b.check_ring_marks(listings["gemm.hip"]) == {}


def _kernel(body):
    return "k:\n" + "\n".join("\t" + l if not l.startswith(".LBB") else l for l in body) + "\n.Lfunc_end0:\n"


def test_ring_marks_count_the_shortest_path():
    mark, load, store, copy = "; ring: 2 loads and stores", "global_load_dwordx4 v[0:3], v4, s[0:1]", "buffer_store_dwordx2 v[0:1], v2, s[0:3], 0 offen", "global_load_lds_dword v2, s[0:1]"
    end = ["; ring: 0 loads and stores", "s_endpgm"]
    assert b.check_ring_marks(_kernel([mark, load, store] + end)) == {"k": 2}
    assert b.check_ring_marks(_kernel([mark, ".LBB0_1:", load, load, mark, store, load, "s_cbranch_scc1 .LBB0_1"] + end)) == {"k": 3}
    for bad in ([mark, load] + end, [mark, load, copy] + end, [mark, "ds_read_b32 v0, v1", load] + end,
                [mark, load, "s_cbranch_scc1 .LBB0_1", store, ".LBB0_1:"] + end,
                [mark, load, load, ".LBB0_1:", mark, load, "s_cbranch_scc1 .LBB0_1", store] + end):
        with pytest.raises(RuntimeError):
            b.check_ring_marks(_kernel(bad))

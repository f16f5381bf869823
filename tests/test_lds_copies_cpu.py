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

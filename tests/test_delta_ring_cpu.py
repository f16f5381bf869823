"""Host-side replay of the output half's copies and waits in the blockwise gated delta rule (chunk_scan_kernel in
csrc/gdn_chunk.hip).

Four wavefronts copy the values and row factors of a sequence's blocks into a ring of kRing slots in LDS, from up to kAhead
blocks ahead, and wait by counts of what they issued since.  Vector-memory operations of a wavefront complete in issue order.
The replay issues copies, loads and stores in the kernel's order, with the counts that its source waits for, and checks:
  * at the wait in block b every copy of block b + 1 is complete (at the first wait: of block 0);
  * no copy is issued to a slot whose block may still be read (block b's is, until block b ends);
  * no count passes what the counter holds.
That the compiler keeps the loads and stores the counts stand on is checked on the generated assembly."""
import os
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_w4a4_block_amd", "csrc", "gdn_chunk.hip")).read()


def constants():
    m = re.search(r"constexpr int kAhead = (\d+), kRing = (\d+);", SRC)
    return int(m.group(1)), int(m.group(2))


def waits(KS):
    """(first, [(blocks below, count)], rest): the counts in the source, evaluated."""
    ahead, _ = constants()
    m = re.search(r"static constexpr int kLoads = (.*?);", SRC)
    names = {"KS": KS, "kAhead": ahead, "kLoads": eval(m.group(1), {"KS": KS})}
    body = SRC[SRC.index("void out_block("):SRC.index("void output()")]
    steps = re.findall(r"if \(turn < (\d+)\)\s*__builtin_amdgcn_s_waitcnt\(vmcnt_imm\((.*)\)\);", body)
    rest = re.search(r"else\s*__builtin_amdgcn_s_waitcnt\(vmcnt_imm\((.*)\)\);", body).group(1)
    first = re.search(r"__builtin_amdgcn_s_waitcnt\(vmcnt_imm\((.*)\)\);\s*// the first block's", SRC).group(1)
    value = lambda text: eval(text, dict(names))  # noqa: E731
    return names["kLoads"], value(first), [(int(n), value(t)) for n, t in steps], value(rest)


def replay(KS, NC, wave, blocks, slack=0):
    """The first violation as a string, or None; every wait lets `slack` more operations stay in flight."""
    ahead, ring = constants()
    loads, first, steps, rest = waits(KS)
    mine = sum(1 for i in range(2 * NC + 2) if i % 4 == wave)          # copies of a block by this wavefront
    issued, held = [], {}                                              # operations in order; slot -> block

    def copy(block, at):
        old = held.get(block % ring)
        if old is not None and old >= at:
            return f"block {block} copied over block {old} in block {at}"
        held[block % ring] = block
        issued.extend([block] * mine)

    def wait(count, block):
        if count > 63:
            return f"a wait for {count}"
        left = issued[max(0, len(issued) - count - slack):] if count + slack else []
        return f"block {block} in flight" if block in left or held.get(block % ring) != block else None

    err = copy(0, 0)
    issued.extend(["load"] * loads)
    err = err or wait(first, 0) or copy(1, 0)
    issued.extend(["load"] * loads)
    for b in range(blocks):
        err = err or (copy(2 * b + 2, b) or copy(2 * b + 3, b) if b < 4 else copy(b + ahead, b))
        err = err or wait(next((c for n, c in steps if b < n), rest), b + 1)
        issued.extend(["load"] * KS + ["store"] + ["load"] * (loads - KS))
        if err:
            return f"KS {KS} NC {NC} wavefront {wave} block {b}: {err}"
    return None


CASES = [(KS, NC, wave) for KS in (2, 4) for NC in (1, 2) for wave in range(4)]


@pytest.mark.parametrize("KS,NC,wave", CASES)
def test_every_wait_covers_the_next_block(KS, NC, wave):
    for blocks in range(1, 40):
        assert replay(KS, NC, wave, blocks) is None


def test_the_replay_sees_a_wait_that_is_too_weak():
    # the first waits have nothing to spare
    assert all(replay(KS, NC, wave, 2, slack=1) for KS, NC, wave in CASES if sum(i % 4 == wave for i in range(2 * NC + 2)) == 1)


def test_the_source_is_the_one_replayed():
    body = SRC[SRC.index("void out_block("):SRC.index("void output()")]
    assert re.search(r"if \(turn < 4\) \{\s*copy_rows\(2 \* b \+ 2\);\s*copy_rows\(2 \* b \+ 3\);\s*\} else \{\s*copy_rows\(b \+ kAhead\);\s*\}", body)
    # the order within a block: mark, copies, wait, Q's loads, the stores, A's loads
    places = [body.index(t) for t in ("ring_mark<LAST ? 0 : kLoads + 1>()", "copy_rows(", "s_waitcnt", "load_q(s", "store_out(s", "load_a(s")]
    assert places == sorted(places)
    body = SRC[SRC.index("void output()"):]
    places = [body.index(t) for t in ("copy_rows(0)", "ring_mark<kLoads>()", "load_q(even", "load_a(even", "ring_mark<0>()", "s_waitcnt", "copy_rows(1)",
                                      "load_q(odd", "load_a(odd", "out_block(even")]
    assert places == sorted(places)
    assert re.search(r"for \(int i = 0; i < 2 \* NC \+ 2; \+\+i\) \{\s*if \(i % 4 != w - 4\) continue;", SRC)

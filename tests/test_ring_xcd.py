"""The ring plan hands pair blocks over within the L2 of one XCD.  CPU model of
the handover between two workgroups of a unit that run on the same or on
different XCDs, and an ISA check that the kernel compares them.

Each XCD has a write-back L2 over one memory.  A line that a workgroup wrote
is written back, and a line that it read is dropped, at any time (an L2 may
evict any of its lines).  The producing workgroup writes a block and then its
flag, both into its L2; the taking one reads the flag from its own L2 until it
is set (or gives up: its waits are bounded) and then the block.  With the
comparison each first posts its XCD, at device scope (into memory), and goes on only
if it reads the other's to be the same."""
import os
import re
import shutil
import subprocess

import pytest

from linear_attention_recurrence_05_amd import build as kbuild
from test_ring_protocol import Violation, _explore, _set

FLAG, BLOCK = 0, 1
ENDS = ("taken", "gave up")


def handover(xcds, compare, start=(None, None)):
    """State: (producer's step, taker's step, memory, posted XCDs, L2s), an L2
    line being (value, dirty) or None; `start` holds what the taker's L2 has of
    the flag's and the block's line before."""

    def read(l2, mem, line):
        """The line's value as an L2 gives it, and the L2 after."""
        if l2[line] is None:
            l2 = _set(l2, line, (mem[line], False))
        return l2[line][0], l2

    def successors(st):
        prod, take, mem, ids, l2s = st
        for x, l2 in enumerate(l2s):                     # any L2 evicts any line
            for line in (FLAG, BLOCK):
                if l2[line] is not None:
                    value, dirty = l2[line]
                    yield (prod, take, _set(mem, line, value) if dirty else mem, ids,
                           _set(l2s, x, _set(l2, line, None)))
        x = xcds[0]
        if prod == "post":
            yield ("block", take, mem, _set(ids, 0, x), l2s)
        elif prod in ("block", "flag"):
            line = BLOCK if prod == "block" else FLAG
            yield ("flag" if prod == "block" else "end", take, mem, ids,
                   _set(l2s, x, _set(l2s[x], line, ("new", True))))
        x = xcds[1]
        if take == "post":
            yield (prod, "compare" if compare else "wait", mem, _set(ids, 1, x), l2s)
        elif take == "compare":
            if None not in ids:
                yield (prod, "wait" if ids[0] == ids[1] else "gave up", mem, ids, l2s)
        elif take == "wait":
            value, l2 = read(l2s[x], mem, FLAG)
            yield (prod, "take" if value == "new" else "wait", mem, ids, _set(l2s, x, l2))
            yield (prod, "gave up", mem, ids, l2s)
        elif take == "take":
            value, l2 = read(l2s[x], mem, BLOCK)
            if value != "new":
                raise Violation(f"the block taken was {value}")
            yield (prod, "taken", mem, ids, _set(l2s, x, l2))

    l2s = [(None, None), (None, None)]
    l2s[xcds[1]] = tuple(v and (v, False) for v in start)
    init = ("post", "post", ("old", "old"), (None, None), tuple(l2s))
    return init, successors, lambda st: st[0] == "end" and st[1] in ENDS


def ends(init, successors, _):
    seen, todo = {init}, [init]
    while todo:
        for st in successors(todo.pop()):
            if st not in seen:
                seen.add(st)
                todo.append(st)
    return {st[1] for st in seen if st[1] in ENDS}


STARTS = [(None, None), ("old", None), (None, "old"), ("old", "old")]


@pytest.mark.parametrize("start", STARTS)
def test_one_xcd_hands_blocks_over(start):
    """(What the unit's one L2 holds of the lines before is what the producer overwrites.)"""
    model = handover((0, 0), True, start)
    assert _explore(*model) > 0
    assert "taken" in ends(*model)


@pytest.mark.parametrize("start", STARTS)
def test_two_xcds_without_the_comparison_take_a_stale_block(start):
    """The flag's line is written back, and read, before the block's."""
    with pytest.raises(Violation, match="the block taken was old"):
        _explore(*handover((0, 1), False, start))


@pytest.mark.parametrize("start", STARTS)
def test_two_xcds_with_the_comparison_give_up(start):
    model = handover((0, 1), True, start)
    assert _explore(*model) > 0
    assert ends(*model) == {"gave up"}


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")
def test_the_kernel_compares_its_units_xcds(tmp_path):
    """The kernel reads the register that names its XCD, posts it and reads the others' at
    device scope, which on gfx950 is the sc1 bit."""
    asm = tmp_path / "k.s"
    subprocess.run([os.environ.get("HIPCC", "hipcc"), *kbuild.source_flags("kda_ring.hip"), "--cuda-device-only", "-S",
                    os.path.join(kbuild.CSRC, "kda_ring.hip"), "-o", str(asm)], check=True, capture_output=True)
    text = asm.read_text()
    kernel = text[text.index("pair_ring_kernel"):]
    at = kernel.find("hwreg(HW_REG_XCC_ID")
    assert at >= 0
    after = kernel[at:]
    post = re.search(r"global_store_dword .* sc1", after)
    assert post and re.search(r"global_load_dword .* sc1", after[post.end():])

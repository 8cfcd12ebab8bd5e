"""A load into LDS takes its LDS address from M0, and the hardware wants one instruction between a scalar write of M0 and
the load that reads it; a vector memory instruction wants five between a vector instruction's write of a scalar register and
its own read of it.  The compiler puts them there for its own loads, but it does not look inside inline assembly, which
is how most kernels here issue loads into LDS.  Every source is compiled with the library's flags to gfx950 assembly, and
neither may occur (CPU only)."""
import os
import re

import pytest

from compiled_sources import HIPCC, all_assembly

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")


def _instructions(lines):
    """The instructions in the order of the text, without labels, directives and comments."""
    for line in lines:
        text = line.split(";")[0].strip()
        if text and not text.startswith((".", "//")) and not text.endswith(":"):
            yield text


def _into_lds(ins):
    return ins.startswith(("global_load_lds", "scratch_load_lds")) or (ins.startswith("buffer_load") and ins.endswith(" lds"))


def _writes_m0(ins):
    return bool(re.match(r"(s_\S+|v_readfirstlane\S*|v_readlane\S*) m0\b", ins))


def loads_without_wait(lines):
    """(write of M0, load) of every load into LDS right behind a write of M0, and the number of loads into LDS."""
    bad, n, last = [], 0, ""
    for ins in _instructions(lines):
        if _into_lds(ins):
            n += 1
            if _writes_m0(last):
                bad.append((last, ins))
        last = ins
    return bad, n


def _scalars(operand):
    m = re.match(r"s(?:(\d+)|\[(\d+):(\d+)\])$", operand)
    return set(range(int(m.group(1) or m.group(2)), int(m.group(1) or m.group(3)) + 1)) if m else set()


def scalars_read_too_early(lines):
    """(write, read) of every scalar register that a vector memory instruction reads within five of its vector write."""
    bad, recent = [], []  # recent: (registers, instruction) of the last five, an s_nop as many as it waits for
    for ins in _instructions(lines):
        op, *args = ins.replace(",", " ").split()
        if op.startswith(("global_", "buffer_", "scratch_", "flat_")):
            used = set().union(*map(_scalars, args)) if args else set()
            bad += [(by, ins) for regs, by in recent[-5:] if regs & used]
        wrote = set()
        if op.startswith(("v_readfirstlane", "v_readlane", "v_cmp")):
            wrote = _scalars(args[0])
        elif op.startswith("v_") and "_co_" in op:
            wrote = _scalars(args[1])
        recent += [(wrote, ins)] * (int(args[0]) + 1 if op == "s_nop" else 1)
        recent = recent[-8:]
    return bad


def test_finds_a_scalar_read_too_early():
    write, load = ["\tv_readfirstlane_b32 s5, v0"], ["\tbuffer_load_dwordx4 v0, s[4:7], s9 offen lds"]
    assert scalars_read_too_early(write + load) and scalars_read_too_early(write + ["\ts_nop 3"] + load)
    assert scalars_read_too_early(["\tv_readfirstlane_b32 s9, v0", "\ts_mov_b32 m0, s3", "\ts_nop 0"] + load)
    assert scalars_read_too_early(["\tv_add_co_u32 v0, s[4:5], v0, v1"] + load)
    assert not scalars_read_too_early(write + ["\ts_nop 4"] + load)
    assert not scalars_read_too_early(["\tv_readfirstlane_b32 s8, v0"] + load)


def test_finds_a_load_without_wait():
    head, load = ["\ts_mov_b32 m0, s3"], ["\tglobal_load_lds_dwordx4 v[0:1], off"]
    assert loads_without_wait(head + load) == ([("s_mov_b32 m0, s3", "global_load_lds_dwordx4 v[0:1], off")], 1)
    assert loads_without_wait(head + [".LBB0_1:", "; comment"] + ["\tbuffer_load_dword v0, s[0:3], s4 offen lds"])[0]
    assert loads_without_wait(head + ["\ts_nop 0"] + load) == ([], 1)
    assert loads_without_wait(head + ["\tglobal_load_dwordx4 v[0:3], v[0:1], off"]) == ([], 0)


@pytest.fixture(scope="module")
def compiled():
    return all_assembly()


def test_no_load_into_lds_follows_a_write_of_m0(compiled):
    total = 0
    for src, lines in compiled.items():
        bad, n = loads_without_wait(lines)
        print("%s: %d loads into LDS, %d without a wait" % (src, n, len(bad)))
        assert not bad, (src, len(bad), bad[:3])
        total += n
    assert total


def test_no_memory_instruction_reads_a_scalar_too_early(compiled):
    for src, lines in compiled.items():
        bad = scalars_read_too_early(lines)
        assert not bad, (src, len(bad), bad[:3])

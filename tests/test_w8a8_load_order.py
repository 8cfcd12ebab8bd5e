"""The tiled W8A8 kernel's k loop, checked on the compiled code (CPU only).

Half way through step kg a wave waits until at most 2 (ST - 2) NSW of its
vector-memory loads are outstanding, and takes that for the arrival of its
loads into LDS of step kg + 1.  That holds if between two of the loop's
barriers there are 2 NSW weight loads into registers and the loads into LDS
come before them: then 2 (ST - 2) NSW weight loads are younger than the loads
into LDS that were issued ST - 2 barriers before.  This test compiles
moe_w8a8_tiled.hip with the library's flags to gfx950 assembly and checks it
in the loop of every instance."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from test_kernel_load_order import misplaced_lds_loads

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def _kernels(lines):
    out, name = {}, None
    for line in lines:
        m = re.match(r"^(_Z\S*k_w8a8_tiled\S*):", line)
        if m:
            name = m.group(1)
            out[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            text = line.split(";")[0].strip()
            if text:
                out[name].append(text)
    return out


def _loops(body):
    """The k loops: single basic blocks that hold a barrier and branch back to their own label."""
    labels = {m.group(1): i for i, x in enumerate(body) for m in [re.match(r"^(\.LBB\w+):", x)] if m}
    found = []
    for i, x in enumerate(body):
        m = re.match(r"^s_(?:c?branch\S*)\s+(\.LBB\w+)", x)
        if m and labels.get(m.group(1), i) < i:
            part = body[labels[m.group(1)]:i + 1]
            if any(p.startswith("s_barrier") for p in part) and not any(p.startswith(".LBB") for p in part[1:]):
                found.append(part)
    return found


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_the_wait_covers_the_loads_into_lds():
    from w4a16_routed_expert_moe_amd import build as b
    d = tempfile.mkdtemp(prefix="moe_asm_")
    try:
        out = os.path.join(d, "tiled.s")
        flags = [f for f in b.FLAGS if f != "-fPIC"] + b.EXTRA.get("moe_w8a8_tiled.hip", [])
        r = subprocess.run([HIPCC] + flags + ["--cuda-device-only", "-S", "-o", out,
                                              os.path.join(b.CSRC, "moe_w8a8_tiled.hip")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        lines = open(out).read().splitlines()
    finally:
        shutil.rmtree(d, ignore_errors=True)
    kernels = _kernels(lines)
    assert len(kernels) >= 10, kernels.keys()
    assert not misplaced_lds_loads(lines)
    seen = 0
    for name, body in kernels.items():
        act, nsw, mc, pf, st, occ = map(int, re.search(r"ILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
        for loop in _loops(body):
            at = [i for i, x in enumerate(loop) if x.startswith("s_barrier")]
            assert len(at) == pf // 2, (name, len(at))  # one barrier per step, pf / 2 steps an iteration
            for n, i in enumerate(at):
                wait = next(x for x in reversed(loop[:i]) if x.startswith("s_waitcnt"))
                m = re.search(r"vmcnt\((\d+)\)", wait)
                assert m and int(m.group(1)) <= 2 * (st - 2) * nsw, (name, wait)
                region = loop[i + 1:at[n + 1]] if n + 1 < len(at) else loop[i + 1:] + loop[:at[0]]
                loads = [x.split()[0] for x in region if x.startswith("global_load")]
                into_lds = [k for k, x in enumerate(loads) if x.startswith("global_load_lds")]
                assert into_lds == list(range(len(into_lds))) and into_lds, (name, loads)
                assert len(loads) - len(into_lds) == 2 * nsw, (name, loads)
                seen += 1
    assert seen >= 2 * len(kernels)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_every_loop_of_every_kernel_is_looked_at():
    """An instance of MC m-tiles has MC / 2 k loops (2, 4, ... MC m-tiles that have rows), of pf / 2 steps each: all of them
    are found, so that the check above leaves none out, and no load into LDS stands in a loop that it does not know."""
    from w4a16_routed_expert_moe_amd import build as b
    d = tempfile.mkdtemp(prefix="moe_asm_")
    try:
        out = os.path.join(d, "tiled.s")
        flags = [f for f in b.FLAGS if f != "-fPIC"] + b.EXTRA.get("moe_w8a8_tiled.hip", [])
        r = subprocess.run([HIPCC] + flags + ["--cuda-device-only", "-S", "-o", out,
                                              os.path.join(b.CSRC, "moe_w8a8_tiled.hip")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        kernels = _kernels(open(out).read().splitlines())
    finally:
        shutil.rmtree(d, ignore_errors=True)
    for name, body in kernels.items():
        act, nsw, mc, pf, st, occ = map(int, re.search(r"ILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
        loops = _loops(body)
        assert len(loops) == mc // 2, (name, len(loops))
        # matrix instructions of a step: two half steps of C m-tiles times nsw subtiles
        products = sorted(sum(x.startswith("v_mfma") for x in loop) for loop in loops)
        assert products == [2 * c * nsw * (pf // 2) for c in range(2, mc + 1, 2)], (name, products)
        # loads into LDS outside the loops: the prologue's ST - 1 steps and the tail's pf / 2 - 1, of every instance
        total = sum(x.startswith("global_load_lds") for x in body)
        inside = sum(x.startswith("global_load_lds") for loop in loops for x in loop)
        per_step = sum(c // 2 for c in range(2, mc + 1, 2))
        assert inside == per_step * (pf // 2) and total - inside == per_step * (st - 1 + pf // 2 - 1), (name, total, inside)

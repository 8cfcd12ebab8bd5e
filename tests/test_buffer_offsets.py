"""A load from a buffer is zeros where its lane offset is not below the buffer's size less the scalar offset: what that says
when the scalar offset itself lies past the end is documented nowhere.  The products in bf16 take the zeros behind the last
row, column or k of a group from that check, and so do the scales of the fp8 products, with buffers that may be shorter
than the tile: their loads carry the whole offset in the lanes and no scalar offset.  (The fp8 codes and weights keep one:
it stays within a row of the former, and the latter's buffers end nowhere.)  Checked on the compiled code (CPU only)."""
import os
import re
import subprocess

import pytest

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")


def _buffer_loads(src, tmp_path):
    from w4a16_routed_expert_moe_amd import build as b
    out = str(tmp_path / "out.s")
    flags = [f for f in b.FLAGS if f != "-fPIC"] + b.EXTRA.get(src, [])
    r = subprocess.run([HIPCC] + flags + ["--cuda-device-only", "-S", "-o", out, os.path.join(b.CSRC, src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # buffer_load_<type> [destination,] lane offset, buffer, scalar offset [offen ...]
    return re.findall(r"(buffer_load_\w+) (?:v\S+, |a\S+, )?(?:v\d+|off), s\[\d+:\d+\], (\S+)", open(out).read())


@pytest.mark.parametrize("src,kind", [("moe_bf16_wide.hip", "buffer_load_dwordx4"), ("moe_bf16_tiled.hip", "buffer_load_dwordx4"),
                                      ("moe_fp8s_tiled.hip", "buffer_load_dword")])
def test_no_scalar_offset(src, kind, tmp_path):
    loads = [s for op, s in _buffer_loads(src, tmp_path) if op == kind]
    assert loads
    other = [s for s in loads if s != "0"]
    assert not other, (len(loads), len(other), other[:5])

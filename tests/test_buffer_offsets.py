"""A load from a buffer is zeros where its lane offset is not below the buffer's size less the scalar offset: what that says
when the scalar offset itself lies past the end is documented nowhere.  The products in bf16 take the zeros behind the last
row, column or k of a group from that check, and so do the scales of the fp8 products, with buffers that may be shorter
than the tile: their loads carry the whole offset in the lanes and no scalar offset.  (The fp8 codes and weights keep one:
it stays within a row of the former, and the latter's buffers end nowhere.)  Checked on the compiled code (CPU only)."""
import os
import re

import pytest

from compiled_sources import HIPCC, assembly

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")


def _buffer_loads(src):
    # buffer_load_<type> [destination,] lane offset, buffer, scalar offset [offen ...]
    return re.findall(r"(buffer_load_\w+) (?:v\S+, |a\S+, )?(?:v\d+|off), s\[\d+:\d+\], (\S+)", "\n".join(assembly(src)))


@pytest.mark.parametrize("src,kind", [("moe_bf16_wide.hip", "buffer_load_dwordx4"), ("moe_bf16_tiled.hip", "buffer_load_dwordx4"),
                                      ("moe_fp8s_tiled.hip", "buffer_load_dword")])
def test_no_scalar_offset(src, kind):
    loads = [s for op, s in _buffer_loads(src) if op == kind]
    assert loads
    other = [s for s in loads if s != "0"]
    assert not other, (len(loads), len(other), other[:5])

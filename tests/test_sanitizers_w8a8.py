"""The host code of the W8A8 and router-balance entry points under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: their HIP sources
built with the sanitizers on the host pass only (the device code is built as
usual and never runs here) and driven by ``tests/host_checks_w8a8.c``, whose
calls are all rejected or have nothing to do.  Everything is built in a
temporary directory."""
import os
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import HIPCC, ROOT, SAN, _run

SOURCES = ["moe_w8a8.hip", "moe_w8a8_tiled.hip", "moe_balance.hip", "moe_combine.hip", "moe_layout.hip"]


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("gcc") is None, reason="hipcc or gcc not found")
def test_host_checks_clean_under_asan_ubsan(tmp_path):
    from w4a16_routed_expert_moe_amd import build as b
    host_san = []
    for flag in ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"]:
        host_san += ["-Xarch_host", flag]

    def compile_one(src):
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        rc, out = _run([HIPCC] + b.FLAGS + ["-O1", "-g"] + host_san + ["-c", os.path.join(b.CSRC, src), "-o", obj])
        assert rc == 0, out
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    drv, exe = str(tmp_path / "checks.o"), str(tmp_path / "checks")
    rc, out = _run(["gcc", "-O1", "-std=c11", "-Wall"] + SAN + ["-I", os.path.join(ROOT, "include"), "-c",
                                                               os.path.join(ROOT, "tests", "host_checks_w8a8.c"),
                                                               "-o", drv])
    assert rc == 0, out
    rc, out = _run([HIPCC, "--offload-arch=gfx950"] + host_san[:4] + ["-o", exe, drv] + objs)
    assert rc == 0, out
    rc, out = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"), timeout=300)
    print(out)
    assert rc == 0 and "runtime error" not in out and "ERROR:" not in out, out

"""The library's HIP sources as gfx950 assembly, compiled once per test run with the library's own flags (CPU only)."""
import functools
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@functools.lru_cache(maxsize=None)
def assembly(src):
    """The lines of one source's assembly."""
    from w4a16_routed_expert_moe_amd import build as b
    d = tempfile.mkdtemp(prefix="asm")
    try:
        out = os.path.join(d, "out.s")
        flags = [f for f in b.FLAGS if f != "-fPIC"] + b.EXTRA.get(src, [])
        r = subprocess.run([HIPCC] + flags + ["--cuda-device-only", "-S", "-o", out, os.path.join(b.CSRC, src)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        with open(out) as f:
            return f.read().splitlines()
    finally:
        shutil.rmtree(d)


def all_assembly():
    """{source: lines} of all of them."""
    from w4a16_routed_expert_moe_amd import build as b
    with ThreadPoolExecutor(max_workers=4) as ex:
        return dict(zip(b.SOURCES, ex.map(assembly, b.SOURCES)))

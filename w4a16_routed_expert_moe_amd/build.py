"""Build ``libmoe_w4a16.so`` (HIP, gfx950) in-tree with hipcc, and ``_bind.so``,
the binding's native argument checks, with g++.  The library needs hipcc only:
where g++ or the headers of Python or torch are missing, the binding's checks
stay in Python.

Every HIP source is compiled for gfx950 only, with packed-fp32 code
generation disabled, and linked into one shared library next to this file.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shlex
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libmoe_w4a16.so")
BIND_PATH = os.path.join(HERE, "_bind.so")
SOURCES = ["moe_route.hip", "moe_permute.hip", "moe_gemm.hip", "moe_gemm_tiled.hip", "moe_down_combine.hip",
           "moe_decode.hip",
           "moe_combine.hip", "moe_layout.hip", "moe_mx_gemm.hip", "moe_gemm_fp4wide.hip",
           "moe_w8a8.hip", "moe_w8a8_tiled.hip", "moe_balance.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]
# per-source additions: both grouped GEMMs keep MFMA results in VGPRs, where
# their scale FMAs read them (in AGPRs every result would be copied back
# first), and both are scheduled for instruction-level parallelism (the
# tiled kernel: every LDS read of a k group issued before the MFMAs that
# consume them; the weight stream: INT4 gate/up at 64 tokens 61.2-61.5% ->
# 62.4-62.7% of HBM, FP4 unchanged), and so is the 512-wide FP4 GEMM
# (prefill8k step 3.24-3.25 -> 3.19 ms, stack43 1.19 -> 1.17 ms); the
# one-launch step, the block-scaled GEMM and the router gained nothing from it
EXTRA = {
    "moe_gemm_fp4wide.hip": ["-mllvm", "-amdgpu-sched-strategy=max-ilp"],
    "moe_gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form", "-mllvm", "-amdgpu-sched-strategy=max-ilp"],
    "moe_gemm_tiled.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form", "-mllvm", "-amdgpu-sched-strategy=max-ilp"],
}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + FLAGS + EXTRA.get(src, []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj


def bind_built_for() -> str:
    """What _bind.so has to be built for to be used in this process."""
    import torch
    return "Python %d.%d, torch %s" % (sys.version_info[0], sys.version_info[1], torch.__version__)


def _compile_bind() -> None:
    import torch
    from torch.utils.cpp_extension import TORCH_LIB_PATH, include_paths
    tmp = BIND_PATH + ".tmp%d" % os.getpid()
    inc = [a for p in include_paths() + [sysconfig.get_paths()["include"]] for a in ("-isystem", p)]
    cmd = shlex.split(os.environ.get("CXX", "g++")) + ["-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-DMOE_BUILT_FOR=\"%s\"" % bind_built_for(),
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] + inc + [
           os.path.join(CSRC, "moe_bind.cpp"), "-o", tmp, "-L", TORCH_LIB_PATH, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for moe_bind.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, BIND_PATH)


def _build_bind() -> bool:
    """Whether the native checks could be built; if not, none of an earlier build are left in their place."""
    try:
        _compile_bind()
        return True
    except (RuntimeError, OSError, ImportError) as e:
        if os.path.exists(BIND_PATH):
            os.remove(BIND_PATH)
        warnings.warn("_bind.so is not built, arguments are checked in Python: %s" % e)
        return False


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        bind = ex.submit(_build_bind)
        objs = list(ex.map(_compile, SOURCES))
        native = bind.result()
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB_PATH)
    if verbose:
        print("built", LIB_PATH, BIND_PATH if native else "")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

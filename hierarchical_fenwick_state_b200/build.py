"""Build libllattn.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m hierarchical_fenwick_state_b200.build [--force]

The library links the CUDA runtime statically, so it loads without a toolkit
on the machine; the output sits next to this file and is what binding.lib()
loads.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["llattn_api.cu", "llattn_simt.cu", "llattn_tc.cu", "llattn_noalloc.cu",
           "llattn_decode.cu", "llattn_bwd.cu", "llattn_bwd_tc.cu", "llattn_gdn.cu",
           "llattn_qknorm.cu", "llattn_glr.cu", "llattn_decode_q8.cu"]
HEADERS = ["llattn_internal.h", "llattn_common.cuh", "llattn_tc_ptx.cuh", "llattn_decode.h",
           "llattn_bwd.h", "llattn_gdn.h", "llattn_qknorm.h", "llattn_glr.h",
           "llattn_decode_q8.h"]
# Built without --use_fast_math: sines of far positions and the 8-bit state's exp at full fp32
# precision, infinities, NaN and denormal values as IEEE has them.  (The recurrence asks for the fast
# exponential by name: its file says what that costs.)
PRECISE = {"llattn_qknorm.cu", "llattn_glr.cu", "llattn_decode_q8.cu"}
LIB = os.path.join(HERE, "libllattn.so")
BUILD_DIR = os.path.join(ROOT, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--use_fast_math",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden", "-Xptxas", "-v",
    "-DLLATTN_BUILD",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "llattn.h"))
    return any(os.path.exists(d) and os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        flags = [f for f in NVCC_FLAGS if not (src in PRECISE and f == "--use_fast_math")]
        cmd = [nvcc(), *flags, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = os.path.join(BUILD_DIR, src + ".log")
        with open(log, "w") as f:
            f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"nvcc failed on {src} (log: {log})")
        if verbose:
            sys.stderr.write(r.stderr)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
           "-cudart", "static", "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libllattn.so failed")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

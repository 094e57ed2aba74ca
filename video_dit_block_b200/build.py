"""Build step of the CUDA library, sm_100a only.

`python -m video_dit_block_b200.build` (or `build()`) compiles csrc/sba.cu and, once for each
pair of row types, csrc/rows.cu, side by side, and links them into libsba.so next to this
file.  (nvcc's own --split-compile gave other registers and spills from one build of the same
source to the next.)
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsba.so")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC"]
ROW_TYPES = [(0, 0), (1, 1), (2, 0), (2, 1), (2, 2)]  # of x and of h: 0 bf16, 1 fp16, 2 fp32


def _sources():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))]
    out.append(os.path.join(ROOT, "include", "sba.h"))
    return out


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or needs_build():
        nvcc = os.environ.get("NVCC", "nvcc")
        tmp = LIB + f".tmp{os.getpid()}"
        units = [("sba.cu", [])] + [("rows.cu", [f"-DROW_X={x}", f"-DROW_H={h}"]) for x, h in ROW_TYPES]
        objects = [f"{tmp}.{i}.o" for i in range(len(units))]
        try:
            running = []
            for (src, defines), obj in zip(units, objects):
                cmd = [nvcc, *NVCC_FLAGS, *defines, "-c", "-o", obj, os.path.join(CSRC, src)]
                if verbose:
                    cmd.insert(1, "-Xptxas=-v")
                running.append((cmd, subprocess.Popen(cmd)))
            failed = [(cmd, p.returncode) for cmd, p in running if p.wait()]
            if failed:
                raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
            subprocess.check_call([nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *objects])
            os.replace(tmp, LIB)
        finally:
            for obj in objects:
                if os.path.exists(obj):
                    os.remove(obj)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

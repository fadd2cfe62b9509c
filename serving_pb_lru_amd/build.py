"""Build libula.so (the HIP engine) for gfx950 with hipcc, in-tree.

Each translation unit compiles in parallel into _build/, then one hipcc link
produces serving_pb_lru_amd/libula.so. Packed FP32 instructions are turned off.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libula.so")
SOURCES = ["k_init.hip", "k_lookup.hip", "k_select.hip", "k_lru.hip", "k_move.hip", "k_gather.hip",
           "k_attend.hip", "k_attend_heads.hip", "k_tree_heads.hip", "k_weigh.hip", "k_rows.hip", "k_norm.hip", "k_entries.hip", "k_lightest.hip",
           "runtime.hip"]

# The attention kernels hold their accumulators in vector registers (vector
# instructions rescale and read them) and what only feeds matrix instructions in
# the accumulation registers; the compiler's default puts them the other way round
# and spills.
EXTRA = {"k_attend.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
         "k_attend_heads.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
         "k_tree_heads.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
         "k_weigh.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r


def build(out: str = OUT, jobs: int = 8) -> str:
    bdir = os.path.join(PKG, "_build")
    os.makedirs(bdir, exist_ok=True)
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(bdir, src.replace(".hip", ".o"))
        objs.append(obj)
        cmds.append([HIPCC, *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj])
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        list(ex.map(_run, cmds))
    tmp = out + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build())
    sys.exit(0)

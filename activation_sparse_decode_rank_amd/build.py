"""Build libsparse_ffn.so (HIP, gfx950 only) in-tree with hipcc.

Usage: python activation_sparse_decode_rank_amd/build.py   (or __graft_entry__.build()).
Run it as a script: importing the package loads the library this builds.
Sources are compiled in parallel into objects under _build/ and linked into the package
directory, where the Python binding loads it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libsparse_ffn.so")
SOURCES = ["sffn_api.hip", "sffn_dispatch.hip", "sffn_stage1.hip", "sffn_decode_b1.hip", "sffn_batch.hip",
           "sffn_mid_bt_h4.hip", "sffn_mid_bt_h8.hip", "sffn_mid_bt_f4.hip", "sffn_mid_bt_f8.hip",
           "sffn_tiles.hip", "sffn_offline.hip", "sffn_measure.hip", "sffn_prefill.hip",
           "sffn_static.hip", "sffn_bundle.hip", "sffn_route.hip", "sffn_i8.hip", "sffn_experts.hip",
           "sffn_experts_api.hip"]
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # packed fp32 instructions are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msgs}")
    if msgs.strip():
        print(msgs, file=sys.stderr)
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()

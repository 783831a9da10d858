"""Build libsparse_ffn.so (HIP, gfx950 only) in-tree with hipcc, and _calls, the extension module that
takes regular calls of mx4.py past ctypes, with the host compiler. That module is for one Python and one
torch, and the package works without it: where it cannot be built, the build says so and goes on.

Usage: python activation_sparse_decode_rank_amd/build.py   (or __graft_entry__.build()).
Run it as a script: importing the package loads the library this builds.
Sources are compiled in parallel into objects under _build/ and linked into the package
directory, where the Python binding loads it.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libsparse_ffn.so")
CALLS = os.path.join(HERE, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
SOURCES = ["sffn_api.hip", "sffn_dispatch.hip", "sffn_stage1.hip", "sffn_decode_b1.hip", "sffn_batch.hip",
           "sffn_mid_bt_h4.hip", "sffn_mid_bt_h8.hip", "sffn_mid_bt_f4.hip", "sffn_mid_bt_f8.hip",
           "sffn_tiles.hip", "sffn_offline.hip", "sffn_measure.hip", "sffn_prefill.hip",
           "sffn_static.hip", "sffn_bundle.hip", "sffn_route.hip", "sffn_i8.hip", "sffn_experts.hip",
           "sffn_experts_api.hip", "sffn_norm.hip", "sffn_norm_f32.hip", "sffn_norm_f16.hip",
           "sffn_norm_bf16.hip", "sffn_mx4.hip", "sffn_mx4_api.hip"]
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CXX = shutil.which("g++") or "g++"

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


def _compile_calls() -> None:
    """_calls against torch's headers; its libraries are the ones that torch has loaded. It carries the
    version of the torch that it is built for."""
    found = importlib.util.find_spec("torch")
    if found is None:
        raise RuntimeError("torch is not installed")
    torch = found.submodule_search_locations[0]
    with open(os.path.join(torch, "version.py"), encoding="utf-8") as f:
        version = re.search(r"^__version__ = ['\"]([\w.+-]+)['\"]", f.read(), re.M)[1]
    inc = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]]
    tmp = CALLS + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", f'-DSFFN_TORCH="{version}"', *(f"-I{i}" for i in inc),
           os.path.join(CSRC, "sffn_calls.cpp"), "-L" + os.path.join(torch, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"sffn_calls.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def build_calls() -> bool:
    """Whether _calls was built. One of an earlier build does not stay: it may not fit the library."""
    try:
        _compile_calls()
        built = CALLS
    except (OSError, RuntimeError, TypeError) as e:  # TypeError: a torch without a version
        print(f"_calls is left out, so calls of mx4.py go through ctypes: {e}", file=sys.stderr)
        built = None
    for old in glob.glob(os.path.join(os.path.dirname(CALLS), "_calls*.so")):
        if old != built:
            os.remove(old)
    return built is not None


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        calls = ex.submit(build_calls)
        objs = list(ex.map(_compile, SOURCES))
        calls = calls.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}" + (f" and {CALLS}" if calls else ""))
    return LIB


if __name__ == "__main__":
    build()

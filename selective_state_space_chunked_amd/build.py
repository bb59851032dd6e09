"""Build the gfx950 shared library libssmscan.so in-tree with hipcc.

Every HIP source under csrc/ and the host library csrc/api.cpp are compiled
for gfx950 and linked into ``selective_state_space_chunked_amd/libssmscan.so``;
the binding's native calls (csrc/pycall.cpp, host code) become ``_pycall.so``
beside it, where torch and the Python headers are installed.
Packed FP32 instructions are disabled for the device code; no fast-math.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libssmscan.so")
PYCALL = os.path.join(PKG, "_pycall.so")
BUILD_DIR = os.path.join(ROOT, "_build")

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
ARCH = os.environ.get("SSMSCAN_ARCH", "gfx950")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + [os.path.join(CSRC, "api.cpp")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [HIPCC, *FLAGS, *lang, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _compile_pycall() -> None:
    """csrc/pycall.cpp against the installed torch and Python headers (host compiler, no GPU code)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    libs = ext.library_paths()[0]
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include")]
    for p in [*ext.include_paths(), sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", p]
    tmp = PYCALL + ".tmp"
    cmd += [os.path.join(CSRC, "pycall.cpp"), "-o", tmp, "-L", libs, f"-Wl,-rpath,{libs}", "-ltorch_python",
            "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling pycall.cpp failed:\n{r.stderr}")
    os.replace(tmp, PYCALL)


def build(verbose: bool = False) -> str:
    """Compiles and links the library, and the native calls where torch and the Python headers are there: the library
    does not need them, nor do its users in C."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        native = ex.submit(_compile_pycall)
        objs = list(ex.map(_compile, srcs))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    try:
        native.result()
    except Exception as e:
        if os.path.exists(PYCALL):   # of an earlier source: its structs may be others by now
            os.remove(PYCALL)
        print(f"{OUT} is built without the native calls: {e}", file=sys.stderr)
    if verbose:
        print(f"built {OUT}")
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

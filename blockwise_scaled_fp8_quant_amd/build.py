"""Build libpuro_fp8.so (gfx950) in-tree with hipcc.

    python blockwise_scaled_fp8_quant_amd/build.py        # or __graft_entry__.build()

(run as a file: importing it through the package would first load the library it builds)

Objects go to <repo>/_build/, the shared library next to this file, and beside it the Python
binding's native marshalling (_marshal.so, host code against torch's headers).  Every HIP source
is compiled with packed-fp32 instruction generation disabled.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpuro_fp8.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
ARCH = "gfx950"

SOURCES = ["quant.hip", "gemm.hip", "gemm_w4.hip", "abi.cpp",
           "norm.hip", "clip.hip", "gemm_rows.hip", "abi_ops.cpp"]


def _hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (expected /opt/rocm/bin/hipcc)")


def _flags(src: str):
    common = ["-O3", "-fPIC", "-std=c++17", "-Wall", "-Wno-unused-function",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if src.endswith(".hip"):
        return common + ["-x", "hip", f"--offload-arch={ARCH}",
                         "-mcode-object-version=5",
                         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    return common + ["-D__HIP_PLATFORM_AMD__"]


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [_hipcc()] + _flags(src) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _torch_dir() -> str:
    """Where torch is installed (found without importing it)."""
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _compile_marshal() -> str:
    """The extension module's object (host code)."""
    torch_include = os.path.join(_torch_dir(), "include")
    obj = os.path.join(OBJDIR, "marshal.cpp.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-fPIC", "-std=c++17", "-Wall", "-I", torch_include,
           "-I", os.path.join(torch_include, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_marshal(obj: str) -> None:
    # torch's libraries are those that importing torch, which comes first, has loaded: no path to them is kept
    tmp = MARSHAL + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-lpuro_fp8", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def build(verbose: bool = True) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-mcode-object-version=5", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_marshal(marshal.result())     # (where torch's headers do not compile, the library is there all the same)
    if verbose:
        print(f"built {LIB} and {os.path.basename(MARSHAL)}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)

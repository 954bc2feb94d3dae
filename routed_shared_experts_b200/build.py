"""Build ``libmoe_b200.so`` (sm_100a) in-tree with nvcc, and with gcc the Python
binding ``_binding`` of its small operators (named for this Python's ABI; without
gcc or Python's headers it is left out, and the calls take the checked path).

    python -m routed_shared_experts_b200.build [--force] [--ptxas-info]

The library is one translation unit (``csrc/block_ops.cu`` includes
``csrc/moe_b200.cu``, and both the kernel headers). The CUDA runtime is linked statically, so loading the library needs
no GPU and no libcuda; the driver API entry point for TMA descriptors is looked
up at run time.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmoe_b200.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
# csrc/binding.c, the Python fast path of the small operators; another Python builds its own beside it
BINDING_PATH = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    out = []
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            if f.endswith((".cu", ".cuh", ".h")):
                out.append(os.path.join(d, f))
    return out


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(s) <= t for s in _sources())


def build_binding(force: bool = False) -> str | None:
    """Path of the binding, or None where it cannot be built: the library does not
    need it."""
    untagged = os.path.join(PKG, "_binding.so")  # any Python would load it
    if os.path.exists(untagged):
        os.remove(untagged)
    src = os.path.join(CSRC, "binding.c")
    if not force and os.path.exists(BINDING_PATH) and os.path.getmtime(src) <= os.path.getmtime(BINDING_PATH):
        return BINDING_PATH
    cc, include = shutil.which("gcc") or shutil.which("cc"), sysconfig.get_paths()["include"]
    if cc is None or not os.path.exists(os.path.join(include, "Python.h")):
        sys.stderr.write("no C compiler or no Python headers: the binding is not built, calls take the checked path\n")
        return None
    res = subprocess.run([cc, "-O2", "-fPIC", "-shared", "-Wall", "-I", include, "-o", BINDING_PATH, src],
                         capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{cc} failed ({res.returncode})")
    return BINDING_PATH


def build(force: bool = False, ptxas_info: bool = False, out: str = LIB_PATH) -> str:
    if out == LIB_PATH:
        build_binding(force)
    if not force and out == LIB_PATH and up_to_date():
        return out
    cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-shared",
           "-cudart", "static", "-I", INCLUDE, "-I", CSRC, "-o", out, os.path.join(CSRC, "block_ops.cu")]
    if ptxas_info:
        cmd[1:1] = ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc failed ({res.returncode})")
    if ptxas_info:
        sys.stderr.write(res.stderr)
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    main()

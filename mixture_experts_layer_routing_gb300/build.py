"""Builds libmoe_gb300.so in-tree from csrc/*.cu for sm_103a with nvcc, and the
tensor binding of its operators, _ops_binding.so, from csrc/ops_binding.cpp.

Each translation unit compiles in its own nvcc process (in parallel), then one
nvcc call links the shared library. A stamp of the sources and flags skips the
build when nothing changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(PKG, "_ops_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _binding_commands() -> tuple:
    """The host compiler's two calls for the binding: against torch's headers, and linked to its libraries and LIB."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cxx = shutil.which("g++") or "c++"
    obj = os.path.join(BUILD, "ops_binding.o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             *[f"-I{p}" for p in inc], "-c", os.path.join(CSRC, "ops_binding.cpp"), "-o", obj],
            [cxx, "-shared", obj, "-o", BINDING + ".tmp", "-L" + os.path.join(root, "lib"), "-ltorch_python",
             "-ltorch_cpu", "-lc10", "-L" + PKG, "-l:libmoe_gb300.so", "-Wl,-rpath,$ORIGIN"])


def _stamp(sources) -> str:
    import torch
    h = hashlib.sha256(" ".join(FLAGS).encode() + torch.__version__.encode())
    for p in sorted(sources + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                    glob.glob(os.path.join(ROOT, "include", "*.h"))):
        h.update(p.encode())
        with open(p, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def build(verbose: bool = False, force: bool = False) -> str:
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    stamp = _stamp(sources)
    stamp_file = LIB + ".stamp"
    if not force and all(map(os.path.exists, (LIB, BINDING, stamp_file))) and open(stamp_file).read() == stamp:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    compile_binding, link_binding = _binding_commands()
    with cf.ThreadPoolExecutor(max_workers=min(9, len(sources) + 1)) as ex:
        binding = ex.submit(subprocess.run, compile_binding, capture_output=True, text=True)
        results = list(ex.map(compile_one, sources))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    for r in (binding.result(), subprocess.run(link_binding, capture_output=True, text=True)):
        if r.returncode != 0:
            raise RuntimeError(f"the binding failed to build:\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))

"""Build the TreeWY CUDA library in-tree: ``libtreewy.so`` beside this file.

Each translation unit under ``csrc/`` is compiled for sm_103a in parallel and
linked with the static CUDA runtime, so the library has no dependency on a
particular libcudart on the loading machine.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtreewy.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]


def nvcc_path() -> str:
    cand = shutil.which("nvcc")
    if cand:
        return cand
    for p in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(p):
            return p
    raise RuntimeError("nvcc not found: the TreeWY library needs the CUDA toolkit to build")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _without_ptxas(log: str) -> str:
    """Warnings without what ptxas says of every kernel."""
    return "".join(x for x in log.splitlines(True) if not re.match(r"ptxas info|\s+\d+ bytes stack frame", x))


def check_launch_registers(src: str, log: str) -> None:
    """``log``: what ptxas -v says of ``src``.  A kernel whose warps hand registers to one another (setmaxnreg) states
    the registers per thread of its launch as kLaunchRegs; one that is compiled to another number would be refused at
    its first launch, since an increase waits for registers that are not there."""
    with open(src) as f:
        stated = re.search(r"\bkLaunchRegs = (\d+)", f.read())
    if stated is None:
        return
    kernel = os.path.basename(src)[:-3] + "_kernel"
    used = {int(n) for name, n in re.findall(r"Compiling entry function '([^']*)'.*?Used (\d+) registers", log, re.S)
            if kernel in name}
    if used != {int(stated.group(1))}:
        raise RuntimeError(f"{kernel} is compiled to {sorted(used)} registers per thread, not {stated.group(1)}: "
                           "its split of registers between warps does not hold with this compiler")


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libtreewy.so."""
    nvcc = nvcc_path()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    hdrs = headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        if not force and not _stale(obj, [src] + hdrs + [__file__]):
            return ""
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj + ".tmp"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
        check_launch_registers(src, res.stderr)
        os.replace(obj + ".tmp", obj)
        return res.stderr if ptxas_verbose else _without_ptxas(res.stderr)

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose or ptxas_verbose:
        for s, log in zip(srcs, logs):
            if log:
                sys.stderr.write(f"== {os.path.basename(s)}\n{log}")
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))

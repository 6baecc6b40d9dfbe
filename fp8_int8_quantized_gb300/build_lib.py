"""Build step of the kvq CUDA library: compiles csrc/*.cu for sm_103a with nvcc
(one process per translation unit, in parallel) and links libkvq.so next to
this file.  Used by ``__graft_entry__.build()`` and by ``python -m
fp8_int8_quantized_gb300.build_lib``."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkvq.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]

# Kernels that deal their launch's registers out among their warpgroups (setmaxnreg) run only with exactly
# these registers per thread; the library refuses to launch another build, this one to make it.
REGISTERS = {"verify_tc_kernel": 96}


def check_registers(text: str) -> None:
    """Raises RuntimeError where a kernel of REGISTERS was compiled to other registers (ptxas -v's report)."""
    for name, used in re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", text, re.S):
        for kernel, want in REGISTERS.items():
            if kernel in name and int(used) != want:
                raise RuntimeError(f"{name}: {used} registers per thread, its warpgroups are dealt {want}")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                     glob.glob(os.path.join(HERE, "..", "include", "*.h")))
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc(), "-Xptxas=-v"] + ARCH + FLAGS + os.environ.get("KVQ_NVCC_FLAGS", "").split() + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        try:
            check_registers(r.stdout + r.stderr)
        except RuntimeError:
            os.remove(cmd[-1])   # the next build compiles it again
            raise
        return r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for out in ex.map(run, jobs):
            if verbose and out:
                print(out)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"], check=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

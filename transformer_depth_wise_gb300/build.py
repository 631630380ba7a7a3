"""Build libattnres.so in-tree: nvcc, sm_103a only, one object per .cu, in parallel.

Usage: ``python -m transformer_depth_wise_gb300.build`` (or ``build()``).
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libattnres.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattnres.so")
    return cand


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_stamp() -> str:
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            p = os.path.join(d, f)
            if os.path.isfile(p):
                h.update(f.encode())
                with open(p, "rb") as fh:
                    h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    return h.hexdigest()


def check_registers(log: str, kernel: str, want: int) -> None:
    """Raise unless ptxas's report (-v) gives every instance of `kernel` exactly `want` registers.

    A kernel whose roles take over registers from one another (setmaxnreg) counts on the number that its launch gives a
    thread; with any other, the host refuses every call.
    """
    used = re.findall(r"Compiling entry function '([^']+)'.*?Used (\d+) registers", log, re.S)
    found = [(name, int(n)) for name, n in used if kernel in name]
    if not found or any(n != want for _, n in found):
        raise RuntimeError(f"{kernel} is planned for {want} registers a thread, ptxas gave {[n for _, n in found]}")


def planned_registers(src: str) -> int:
    """kRegs of a source file: the registers a thread that its roles' shares start from."""
    with open(src) as fh:
        return int(re.search(r"constexpr int kRegs = (\d+);", fh.read()).group(1))


# Sources with a kernel of register shares.
REGISTER_SHARES = {"linear_tc.cu": "linear_tc_kernel"}


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile every csrc/*.cu for sm_103a and link libattnres.so; returns its path."""
    stamp_file = os.path.join(OBJDIR, "stamp")
    stamp = _deps_stamp()
    if not force and os.path.exists(LIB) and os.path.exists(stamp_file):
        with open(stamp_file) as fh:
            if fh.read().strip() == stamp and not extra_flags:
                return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        shares = REGISTER_SHARES.get(os.path.basename(src))
        cmd = [cc, *ARCH, *flags, *(["-Xptxas", "-v"] if shares else []), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if shares:
            check_registers(r.stdout + r.stderr, shares, planned_registers(src))
        if verbose and (r.stdout or r.stderr) and (extra_flags or not shares):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    xflags = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=force or bool(xflags), verbose=True, extra_flags=xflags))

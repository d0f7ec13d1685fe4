"""Build the CUDA library libgm_b200.so (sm_100a) next to this file.

    python -m sparse_dynamic_routing_b200.build [--force] [--verbose]

Two translation units (csrc/gm_api.cu, csrc/gm_attn.cu), compiled side by side, with the C ABI
of include/gm.h (--checked builds the variant that verifies every input edge tensor,
libgm_b200_checked.so); an object is compiled again when a file it includes is newer. The CUDA
runtime is
linked statically, so the library only needs the NVIDIA driver at run time. No fast-math:
the referral step relies on IEEE fp32 products and sums (it uses the _rn intrinsics), and
denormals are kept (-ftz=false).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import threading
import time

SELF = os.path.abspath(__file__)
HERE = os.path.dirname(SELF)
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgm_b200.so")
# the checked build: every call first verifies the edge tensors it reads (GM_CHECKED=1)
CHECKED_LIB = os.path.join(HERE, "libgm_b200_checked.so")
HEADER = os.path.join(ROOT, "include", "gm.h")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-Xcompiler", "-fPIC", "-cudart", "static",
]
OBJ_DIR = os.path.join(HERE, "build")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [HEADER])


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in [*sources(), SELF])


def _object_is_stale(obj: str, dep: str) -> bool:
    """Whether an object is older than this file (its flags) or than a file named in its dependency list
    (as nvcc wrote it)."""
    if not os.path.exists(obj) or not os.path.exists(dep):
        return True
    t = os.path.getmtime(obj)
    with open(dep) as f:
        files = f.read().split(":", 1)[-1].replace("\\\n", " ").split()
    return any(not os.path.exists(x) or os.path.getmtime(x) > t for x in [*files, SELF])


class _Compile:
    """The object of one source: up to date, or on its way in a compiler process of its own. The
    compiler writes under names that no other build uses; a whole object takes its place by renaming."""

    def __init__(self, src: str, variant: str, flags: list[str], force: bool):
        self.obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + variant + ".o")
        self.proc = None
        if force or _object_is_stale(self.obj, self.obj + ".d"):
            self.start = time.time()
            self.tmp = f"{self.obj}.{os.getpid()}.{threading.get_ident()}.tmp"
            self.proc = subprocess.Popen([nvcc(), *NVCC_FLAGS, *flags, "-MD", "-MF", self.tmp + ".d", "-c", src,
                                          "-o", self.tmp])

    def finish(self) -> None:
        """Waits for the compiler; raises if it failed."""
        if self.proc is None:
            return
        try:
            if self.proc.wait() != 0:
                raise subprocess.CalledProcessError(self.proc.returncode, self.proc.args)
            # as old as its sources were when they were read: an edit made meanwhile is newer
            os.utime(self.tmp, (self.start, self.start))
            os.replace(self.tmp + ".d", self.obj + ".d")
            os.replace(self.tmp, self.obj)
        finally:
            for left in (self.tmp, self.tmp + ".d"):
                if os.path.exists(left):
                    os.remove(left)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    lib = CHECKED_LIB if checked else LIB
    if force or stale(lib):
        os.makedirs(OBJ_DIR, exist_ok=True)
        start = time.time()
        flags = (["-DGM_CHECKED=1"] if checked else []) + (["-Xptxas", "-v"] if verbose else [])
        made = [_Compile(src, "_checked" if checked else "", flags, force)
                for src in sorted(glob.glob(os.path.join(CSRC, "*.cu")))]
        failed = None
        for m in made:  # every compiler has ended before a failure is passed on
            try:
                m.finish()
            except subprocess.CalledProcessError as e:
                failed = failed or e
        if failed is not None:
            raise failed
        tmp = os.path.join(OBJ_DIR, f"{os.path.basename(lib)}.{os.getpid()}.{threading.get_ident()}.tmp")
        try:
            subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", *(m.obj for m in made), "-o", tmp], check=True)
            os.utime(tmp, (start, start))
            os.replace(tmp, lib)
        finally:
            if os.path.exists(tmp):
                os.remove(tmp)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
                checked="--checked" in sys.argv))

"""Builds the HIP library ``libets_topk.so`` in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", name) for name in
           ("ets_topk.hip", "ets_rope_cache.hip", "ets_scores.hip", "ets_attend.hip", "ets_attend_wide.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libets_topk.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # packed fp32 instructions are disabled for every HIP source of this library
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # LDS histogram atomics are aggregated by hand; keep the compiler from
    # rewriting them into wave reductions
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose: bool = False) -> str:
    """Compile the library (always, the sources side by side) and return its path."""
    work = tempfile.mkdtemp(prefix="ets_build_")
    try:
        running = []
        for src in SOURCES:
            obj = os.path.join(work, os.path.basename(src) + ".o")
            cmd = [hipcc(), *(f for f in HIPCC_FLAGS if f != "-shared"), "-c", "-I", INCLUDE, src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            log = open(obj + ".log", "w+")
            running.append((obj, log, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT)))
        failed = ""
        for obj, log, child in running:
            if child.wait() != 0:
                log.seek(0)
                failed += log.read()
            log.close()
        if failed:
            raise RuntimeError("hipcc failed:\n" + failed)
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *(obj for obj, _, _ in running), "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
        os.replace(tmp, LIB)
    finally:
        shutil.rmtree(work, ignore_errors=True)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))

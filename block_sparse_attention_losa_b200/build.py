"""Builds liblosa.so in-tree with nvcc for sm_100a.

    python block_sparse_attention_losa_b200/build.py   (or build())

The library is plain C ABI (include/losa.h) over CUDA kernels; it links the
CUDA runtime statically and resolves the driver's tensor-map encoder at run
time, so it needs no libcuda at link time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblosa.so")
OBJ = os.path.join(HERE, "_build")
SOURCES = ["losa_api.cu", "losa_attention.cu", "losa_select.cu", "losa_rope.cu",
           "losa_backward.cu", "losa_backward_mma.cu"]
HEADERS = ["losa_device.cuh", "losa_attention.cuh", "losa_cut.cuh", "losa_internal.h"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(path: str, deps) -> bool:
    """Whether `path` exists and is newer than every dependency."""
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path)
                                        for d in deps)


def _compile(src: str, force: bool) -> str:
    """Compiles one source (unless its object is current) and returns the
    object; the compiler's log is kept beside it."""
    obj = os.path.join(OBJ, src.replace(".cu", ".o"))
    deps = [os.path.join(CSRC, f) for f in [src] + HEADERS]
    deps += [os.path.join(ROOT, "include", "losa.h"), os.path.abspath(__file__)]
    if not force and _newer(obj, deps) and os.path.exists(obj + ".log"):
        return obj
    tmp = f"{obj}.{os.getpid()}.tmp"
    cmd = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-Xptxas", "-v",
           "-I", os.path.join(ROOT, "include"), "-c", "-o", tmp, os.path.join(CSRC, src)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    with open(obj + ".log", "w") as f:
        f.write(res.stderr)
    os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps += [os.path.join(ROOT, "include", "losa.h"), os.path.abspath(__file__)]
    if not force and _newer(LIB, deps):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = list(pool.map(lambda src: _compile(src, force), SOURCES))
    log = ""
    for obj in objects:
        with open(obj + ".log") as f:
            log += f.read()
    if verbose:
        sys.stderr.write(log)
    check_attention_registers(log)
    out_tmp = LIB + ".tmp"
    res = subprocess.run([nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                          "-Xcompiler", "-fPIC", "-o", out_tmp] + objects,
                         capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout + res.stderr)
    os.replace(out_tmp, LIB)
    return LIB


def check_attention_registers(ptxas_log: str, want: int = 168) -> None:
    """The attention kernels, forward and backward, split their launch
    registers between warpgroups with setmaxnreg; the split adds up only if every instance
    launches with exactly `want` registers per thread (else a warpgroup
    would wait for registers that never come). Refuse the build otherwise."""
    current, seen = None, 0
    for line in ptxas_log.splitlines():
        if "Compiling entry function" in line:
            current = any(k in line for k in ("attn_kernel", "bwd_tiles_kernel"))
        elif current and "Used" in line and "registers" in line:
            used = int(line.split("Used")[1].split("registers")[0])
            seen += 1
            if used != want:
                raise RuntimeError(f"attention kernel launches with {used} registers, "
                                   f"the setmaxnreg split assumes {want}")
    if seen == 0:
        raise RuntimeError("no attention kernel found in the ptxas log")


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

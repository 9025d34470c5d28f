"""Build libtp.so (the C-ABI CUDA library) in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process, in parallel, then
linked into one shared library next to this file.  Usage (run it as a
script: importing the package needs the library it builds)::

    python tensor_sharded_linear_tp_gb300/build.py [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libtp.so")
SOURCES = ["tp_host.cu", "tp_copy.cu", "tp_gemm.cu", "tp_attention.cu", "tp_flash.cu", "tp_quant.cu", "tp_fp8.cu",
           "tp_kv_append.cu", "tp_paged_attention.cu", "tp_paged_tiles.cu", "tp_safetensors.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Kernels whose warpgroups share the block's registers out among themselves: the launch has to have this many a thread.
REGISTERS = {"tp_paged_tiles.cu": ("paged_tiles_kernel", 128)}


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _flags(verbose: bool) -> list[str]:
    f = ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _newest_input_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def up_to_date() -> bool:
    return os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= _newest_input_mtime()


def check_registers(src: str, log: str) -> None:
    """Raise unless ptxas gave every instance of the source's kernel the registers that its split adds up to."""
    if src not in REGISTERS:
        return
    kernel, want = REGISTERS[src]
    used = re.findall(r"Compiling entry function '[^']*" + kernel + r"[^']*'.*?Used (\d+) registers", log, re.S)
    if not used or any(int(n) != want for n in used):
        raise RuntimeError(f"{src}: {kernel} needs {want} registers a thread, ptxas gave {used or 'no report'}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libtp.so if any source is newer than it; return its path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = _flags(verbose)

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        report = [] if verbose or src not in REGISTERS else ["-Xptxas", "-v"]
        cmd = [nvcc, *flags, *report, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        check_registers(src, r.stdout + r.stderr)
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/shared-memory usage")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()

"""Build libkvq.so (the C-ABI CUDA library) in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process, in parallel, then
linked into ``rotated_int2_kv_kvq_gb300/libkvq.so``.  The output is git-ignored
and rebuilt on every machine (the library is architecture specific)."""
from __future__ import annotations

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkvq.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]

# Kernels whose launch needs an exact register count: source -> (kernel, registers a thread,
# instantiations).  prefill_kernel's roles share out what the block was launched with, so with
# any other count the call would be refused at run time.
REGISTERS = {"kvq_prefill.cu": ("prefill_kernel", 128, 2)}


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvq.so")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def check_registers(source: str, ptxas_log: str) -> None:
    """Raise if the compiler gave a kernel of REGISTERS another register count than it needs."""
    name, want, count = REGISTERS[os.path.basename(source)]
    got = []
    for entry in ptxas_log.split("Compiling entry function")[1:]:
        used = re.search(r"Used (\d+) registers", entry)
        if used and re.search(r"\d" + name + r"(?![a-z_])", entry.split("'")[1]):
            got.append(int(used.group(1)))
    if got != [want] * count:
        raise RuntimeError(f"{source}: {name} needs {want} registers a thread in each of {count} "
                           f"instantiations, the compiler used {got}")


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        exact = os.path.basename(src) in REGISTERS
        if ptxas_verbose or exact:
            cmd.insert(1, "-Xptxas=-v")
        if verbose:
            print(" ".join(cmd))
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if exact:
            check_registers(src, r.stderr)
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(compile_one, srcs))
    if ptxas_verbose:
        for _, err in results:
            print(err)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))

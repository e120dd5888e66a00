"""Compile libss.so (the sm_103a CUDA kernels + C ABI) in-tree with nvcc.

The translation units compiled in parallel, one -gencode (sm_103a), no cmake; the output goes to
speculative_verification_gb300/_build/libss.so.
"""
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libss.so")
SOURCES = ["ss_kernel.cu", "ss_hist.cu", "ss_shard.cu", "ss_fused.cu", "ss_cache.cu", "ss_attn.cu",
           "ss_attn_bf16.cu", "ss_attn_int4.cu"]
SHARED_REGISTERS = ["ss_attn_bf16.cu", "ss_attn_int4.cu"]  # whose kernels' warpgroups share registers out again
DEPS = SOURCES + ["ss_hist.h", "ss_cache.h", "ss_attn.cuh", "ss_philox.cuh", "ss_ptx.cuh", "ss_nvtx.h"]

NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-Xcompiler", "-fPIC",
]
LINK_FLAGS = ["-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-ldl"]


def nvcc():
    cand = os.environ.get("NVCC") or os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def check_registers(log):
    """ptxas's report of the attention kernels: where warpgroups share out the
    launch's registers again, the compiler has to have used the number per
    thread that the shares are made of (it is in the kernel's name; with fewer
    a warpgroup would wait for ever, so the launch would be refused)."""
    found = re.findall(r"entry function '_ZN3ssa11attn_kernelILi(\d+)ELb([01])ELi(\d+)ELi(\d+)E[^']*'"
                       r".*?Used (\d+) registers", log, flags=re.S)
    if not found:
        raise RuntimeError("no attention kernel in the compiler's report")
    for rows, packed, halves, want, used in found:
        if int(want) and want != used:
            raise RuntimeError("attention kernel for %s rows, %s, %s x 64 channels: the compiler used %s registers per "
                               "thread, its warpgroups share out %s" %
                               (rows, "4 bits" if packed == "1" else "bf16", halves, used, want))


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    inputs = [os.path.join(CSRC, d) for d in DEPS] + [os.path.join(INCLUDE, "ss.h")]
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= max(map(os.path.getmtime, inputs)):
        return LIB
    # one object per translation unit, compiled in parallel, then one link
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc()] + NVCC_FLAGS + ["-I" + INCLUDE, "-c", "-o", obj, os.path.join(CSRC, src)]
        checked = src in SHARED_REGISTERS
        if verbose or checked:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stderr=subprocess.PIPE if checked else None, text=True)))
        objs.append(obj)
    logs = {src: p.communicate()[1] for src, p in procs}
    failed = [src for src, p in procs if p.returncode != 0]
    for src, log in logs.items():
        if log and (verbose or src in failed):
            sys.stderr.write(log)
    if failed:
        raise subprocess.CalledProcessError(1, "nvcc " + " ".join(failed))
    for src in SHARED_REGISTERS:
        check_registers(logs[src])
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([nvcc()] + LINK_FLAGS + ["-o", tmp] + objs)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))

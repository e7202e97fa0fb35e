"""Build libkv2.so in-tree for sm_100a (nvcc, no JIT cache).

    python -m bit_kv_cache_centroid_b200.build [--force]
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkv2.so")
SOURCES = ["api.cu", "quantize.cu", "quantize_rows.cu", "decode.cu", "decode_groups.cu", "decode_noalloc.cu", "fit.cu", "chunk.cu", "fit_centroids.cu", "top1.cu",
           "rows_attn.cu", "rotary.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _newer(src_paths, target):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in src_paths)


# Registers per thread that a kernel trades between its warps at run time
# (``RCfg::kRegs`` in rows_attn.cu): its launch refuses any other number.
TRADED = {"rows_attn.cu": ("rows_attn_kernel", 72)}


def wrong_registers(src: str, log: str) -> list:
    """(kernel, registers) of ptxas -v's log whose number is not the traded one."""
    name, want = TRADED[src]
    used = re.findall(r"Compiling entry function '([^']*)'.*?Used (\d+) registers", log, re.S)
    return [(k, int(n)) for k, n in used if name in k and int(n) != want]


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "kv2.h"))
    objs, jobs = [], []
    for src in SOURCES:
        sp = os.path.join(CSRC, src)
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _newer([sp] + headers, obj):
            cmd = [NVCC, "-c", sp, "-o", obj + ".tmp"] + FLAGS
            if verbose or src in TRADED:
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append((cmd, src, obj))

    def compile_one(job):
        cmd, src, obj = job
        if src in TRADED:
            r = subprocess.run(cmd, stderr=subprocess.PIPE, text=True)
            if verbose or r.returncode:
                print(r.stderr, file=sys.stderr, flush=True)
            r.check_returncode()
            for kernel, n in wrong_registers(src, r.stderr):
                print(f"warning: {src}: {kernel} takes {n} registers, its role split {TRADED[src][1]}: "
                      "its calls will return KV2_ERR_CUDA", file=sys.stderr, flush=True)
        else:
            subprocess.run(cmd, check=True)
        os.replace(obj + ".tmp", obj)

    # the translation units are independent: compile them side by side
    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as pool:
        for f in [pool.submit(compile_one, j) for j in jobs]:
            f.result()
    if force or _newer(objs, LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([NVCC, "-shared", "-o", tmp] + objs +
                       ["-gencode", "arch=compute_100a,code=sm_100a"], check=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

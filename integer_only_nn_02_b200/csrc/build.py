"""Build libict.so (sm_100a) in-tree with nvcc.

Usage: python -m integer_only_nn_02_b200.csrc.build [--force]
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
LIB = os.path.join(PKG, "libict.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
SOURCES = ["ict_api.cu", "ict_attention.cu", "ict_norm.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-warn-spills",
]


def dependencies() -> list:
    """Every file the library is built from: the sources and headers in this directory,
    the public headers, and this script."""
    deps = [os.path.join(HERE, f) for f in sorted(os.listdir(HERE)) if f.endswith((".cu", ".cuh", ".h"))]
    deps += [os.path.join(INCLUDE, f) for f in sorted(os.listdir(INCLUDE)) if f.endswith(".h")]
    return deps + [os.path.abspath(__file__)]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in dependencies())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the sources at the same time, one object each, and links them."""
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    objs = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    cmds = [[NVCC, *FLAGS, *(["-Xptxas=-v"] if verbose else []), "-c", "-o", o, os.path.join(HERE, f)]
            for o, f in zip(objs, SOURCES)]
    try:
        procs = []
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd))
            procs.append(subprocess.Popen(cmd))
        codes = [p.wait() for p in procs]
        for cmd, code in zip(cmds, codes):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.run([NVCC, *FLAGS, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

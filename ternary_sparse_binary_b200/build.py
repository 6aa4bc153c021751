"""Build libwal.so in-tree with nvcc for sm_100a (B200)."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libwal.so")
SOURCES = ["wal_host.cpp", "wal_gemv.cu", "wal_stream.cu", "wal_body.cu", "wal_tc.cu", "wal_noalloc.cu", "wal_pq2.cu", "wal_base3.cu", "wal_rc1.cu", "wal_head.cu", "wal_cache.cu", "wal_qkv.cu", "wal_plan.cu", "wal_attn.cu", "wal_attn_ring.cu", "wal_attn_tc.cu"]
HEADERS = ["wal_internal.h", "wal_device.cuh", "wal_stream.h", "wal_ptx.cuh", "wal_tc.h", "wal_kv.h", "wal_rope.cuh", "wal_attn.h", "wal_attn_dec.cuh", os.path.join("..", "..", "include", "wal.h")]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo", "--threads", "8",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fopenmp",
    "-shared",
]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [__file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *[os.path.join(CSRC, s) for s in SOURCES], "-o", tmp, "-lgomp"]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd, cwd=CSRC)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))

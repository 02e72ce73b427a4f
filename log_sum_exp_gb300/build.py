"""Build liblse.so in-tree for sm_103a (nvcc; one process per translation unit)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD, "liblse.so")

SOURCES = ["lse_api.cu", "lse_kernels_f32.cu", "lse_kernels_bf16.cu", "lse_kernels_f16.cu",
           "lse_logprob_f32.cu", "lse_logprob_bf16.cu", "lse_logprob_f16.cu", "lse_backward.cu",
           "lse_strided.cu", "lse_rowtile.cu", "lse_noalloc.cu", "lse_ex16_f32.cu",
           "lse_ex16_bf16.cu", "lse_ex16_f16.cu", "lse_stats.cu", "lse_stats_f32.cu", "lse_stats_bf16.cu",
           "lse_stats_f16.cu", "lse_grads.cu", "lse_embed.cu"]
HEADERS = ["lse_device.cuh", "lse_edges.cuh", "lse_kernels.cuh", "lse_internal.h", "lse_elem.cuh", "lse_topk.cuh",
           "lse_stats.cuh", "lse_stats_common.cuh"]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _cuda_lib_dir() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return os.path.join(home, "lib64")


def _mtime(path: str) -> float:
    return os.path.getmtime(path) if os.path.exists(path) else -1.0


def _stale() -> bool:
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps += [os.path.join(INCLUDE, "lse.h"), os.path.abspath(__file__)]
    newest = max(_mtime(p) for p in deps)
    return _mtime(LIB_PATH) < newest


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit in parallel and link liblse.so."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            print(res.stdout + res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", f"-rpath,{_cuda_lib_dir()}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))

"""Build libmesh_attn.so in-tree with nvcc for sm_103a (no cmake, one -gencode).

Each translation unit compiles in parallel into _build/, then one nvcc link step writes
tiled_distributed_attention_gb300/libmesh_attn.so (CUDA runtime linked statically, so the
library loads on a machine without a GPU; the driver is reached at run time).  Beside them g++
builds _binding.so, the package's part that takes tensors, against the installed PyTorch.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmesh_attn.so")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["planner.cpp", "abi.cu", "tile_fwd_tc.cu", "tile_fwd_tc32.cu", "merge.cu", "noalloc.cu",
           "tile_bwd_simt.cu", "tile_bwd_tc.cu", "bwd_aux.cu", "rope.cu", "diff_abi.cu", "diff_aux.cu", "diff_fwd_tc.cu",
           "diff_bwd_tc.cu", "diff_bwd_tc32.cu", "diff_decode.cu", "paged_append.cu", "paged_rows.cu", "score_abi.cu",
           "score_fwd.cu", "score_fwd_64.cu", "score_fwd_128.cu", "score_fwd_paged_64.cu", "score_fwd_paged_128.cu",
           "score_bwd.cu", "score_bwd_64.cu", "score_bwd_128.cu", "score_simt.cu"]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmesh_attn.so")


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
           *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd.insert(1, "-x")
        cmd.insert(2, "cu")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_binding() -> None:
    import torch  # its headers and libraries, of the very version that will load the module
    at = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    include = [INCLUDE, os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], cuda]
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-shared", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for d in include for x in ("-isystem" if at in d else "-I", d)), os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(lambda s: _compile(s, list(extra)), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    binding.result()  # after the library, which does not need it
    return LIB


if __name__ == "__main__":
    build(verbose=True)

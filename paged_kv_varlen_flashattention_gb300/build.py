"""Builds libpa_varlen.so in-tree with nvcc for sm_103a (one -gencode, translation
units compiled in parallel, then linked with the static CUDA runtime), and beside it the
binding's CPython module, which reads tensors of the installed torch."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa_varlen.so")

SOURCES = ["api.cpp", "errword.cu", "splitkv_bf16.cu", "splitkv_f16.cu", "prefill_tc.cu", "decode_tc.cu", "noalloc.cu",
           "kv_append.cu", "padded.cu", "rope_append.cu", "q8_append.cu",
           "q8_bf16.cu", "q8_f16.cu", "prefill_q8.cu", "prefill_q8_wide.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def tensor_args_path() -> str:
    """The binding's module, built for one version of torch and of Python."""
    import torch
    return os.path.join(PKG, f"_pa_tensor_args-{torch.__version__}-{sysconfig.get_config_var('SOABI')}.so")


def build_tensor_args(path: str) -> None:
    import torch
    home = os.path.dirname(torch.__file__)
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
           os.path.join(CSRC, "tensor_args.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on tensor_args.cpp:\n{r.stderr[-6000:]}")
    os.replace(tmp, path)


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _flags():
    return ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC] + ARCH


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(tensor_args_path()):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(tensor_args_path()))
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if os.path.getmtime(os.path.join(d, f)) > t:
                return True
    return False


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc()] + _flags() + list(extra_flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr[-6000:]}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        module = ex.submit(build_tensor_args, tensor_args_path())
        objs = list(ex.map(compile_one, SOURCES))
        module.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

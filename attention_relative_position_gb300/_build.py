"""Builds libfatattn.so (the CUDA library behind include/fat_attn.h) in-tree with nvcc for
sm_103a. Translation units compile in parallel; the link uses nvcc with the static CUDA runtime. The
extension module of the paged-cache calls is compiled beside them with g++ against torch's headers."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libfatattn.so")
SOURCES = ["fat_attn_api.cu", "fat_attn_fwd.cu", "fat_attn_bwd.cu", "fat_attn_decode.cu",
           "fat_attn_noalloc.cu", "fat_rope.cu", "fat_norm_ce.cu", "fat_paged_maps.cu",
           "fat_paged_attn.cu", "fat_paged_few.cu", "fat_paged_tile.cu"]
HEADERS = ["sm103_ptx.cuh", "fat_attn_internal.cuh", "fat_paged.cuh"]
PUBLIC_HEADERS = [os.path.join(ROOT, "include", h) for h in ("fat_attn.h", "fat_attn_debug.h")]
BINDING = "paged_binding.cpp"
CALLS_PATH = os.path.join(PKG, "_paged_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfatattn.so")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, log_dir: str) -> str:
    obj = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
    deps = [os.path.join(CSRC, src)] + [os.path.join(CSRC, h) for h in HEADERS] + PUBLIC_HEADERS
    if not _stale(obj, deps):
        return obj
    cmd = [nvcc()] + ARCH + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, src + ".log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr[-4000:]}")
    return obj


def _compile_binding() -> str:
    """_paged_calls.so: a Python extension module that calls the library's C ABI."""
    src = os.path.join(CSRC, BINDING)
    if not _stale(CALLS_PATH, [src] + PUBLIC_HEADERS):
        return CALLS_PATH
    import sysconfig

    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{base}/include", f"-I{base}/include/torch/csrc/api/include", f"-I{cuda}/include",
           f"-I{sysconfig.get_paths()['include']}", src, "-o", tmp, f"-L{base}/lib", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ldl"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(OBJ_DIR, BINDING + ".log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING}:\n{res.stderr[-4000:]}")
    os.replace(tmp, CALLS_PATH)
    return CALLS_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    if force:
        for s in SOURCES:
            o = os.path.join(OBJ_DIR, s.replace(".cu", ".o"))
            if os.path.exists(o):
                os.remove(o)
        if os.path.exists(CALLS_PATH):
            os.remove(CALLS_PATH)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, OBJ_DIR), SOURCES))
        calls.result()
    if force or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr[-4000:]}")
        os.replace(tmp, LIB_PATH)
    if verbose:
        for s in SOURCES:
            p = os.path.join(OBJ_DIR, s + ".log")
            if os.path.exists(p):
                print(open(p).read())
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))

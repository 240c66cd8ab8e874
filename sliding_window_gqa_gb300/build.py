"""Builds libwa.so in-tree with nvcc for sm_103a (one translation unit per job, in parallel), and the binding's
wa_bind.so, a Python extension against the installed PyTorch's headers, with g++ at the same time.  Without wa_bind.so
every call still works, so where it cannot be built that is said and the build goes on."""
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
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libwa.so")
BIND = os.path.join(OUT, "wa_bind.so")
SOURCES = ["wa_api.cu", "wa_decode.cu", "wa_prompt.cu", "wa_rerun.cu", "wa_static.cu", "wa_decode_tc.cu", "wa_prep.cu", "wa_prompt_sparse.cu",
           "wa_tree.cu", "wa_tree_verify.cu", "wa_tree_commit.cu", "wa_paged_append.cu",
           "wa_paged.cu"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwa.so")
    return cand


def _compile(nvcc: str, src: str, extra) -> str:
    obj = os.path.join(OUT, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_bind(nvcc: str, torch_dir: str) -> str:
    import torch
    obj = os.path.join(OUT, "wa_bind.o")
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
           os.path.join(ROOT, "include")]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    built_for = f"PyTorch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", f'-DWA_BIND_FOR="{built_for}"',
          *[f"-I{p}" for p in inc], "-c", os.path.join(CSRC, "wa_bind.cpp"), "-o", obj], "g++ on wa_bind.cpp")
    return obj


def build(verbose: bool = False, extra=()) -> str:
    """Compile every source and link libwa.so and wa_bind.so; returns libwa.so's path."""
    import torch
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()
    torch_dir = os.path.dirname(torch.__file__)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(_compile_bind, nvcc, torch_dir)
        objs = list(ex.map(lambda s: _compile(nvcc, s, list(extra)), SOURCES))
        try:
            bind_obj, bind_error = bind.result(), None
        except Exception as e:
            bind_obj, bind_error = None, e
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    try:
        if bind_error:
            raise bind_error
        tmp = BIND + ".tmp"
        _run(["g++", "-shared", "-o", tmp, bind_obj, "-L" + OUT, "-l:libwa.so", "-L" + os.path.join(torch_dir, "lib"),
              "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], "link of wa_bind.so")
        os.replace(tmp, BIND)
    except Exception as e:
        if os.path.exists(BIND):        # an earlier build's, of other sources
            os.remove(BIND)
        print(f"wa_bind.so was not built, the drafted-token and paged-cache calls go through ctypes: {e}", file=sys.stderr)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])

"""Builds libpkv.so in-tree for sm_103a with nvcc (no cmake), and beside it the
extension module that passes torch tensors to some of its calls.

The translation units compile in parallel; the CUDA runtime is linked
statically, so the library depends only on the driver at run time.  The module
is compiled against the installed torch's headers.
Usage: python -m paged_kv_cache_311_gb300.build [--verbose-ptxas]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB_DIR = os.path.join(HERE, "_lib")
SOURCES = ["pkv_abi.cu", "pa_decode_f32.cu", "pa_decode_f16.cu", "pa_decode_bf16.cu",
           "pkv_static_ws.cu", "pkv_plan.cu", "pkv_usage.cu", "pkv_block_pool.cu",
           "q8_cache.cu", "block_select.cu", "list_attention.cu", "q4_cache.cu", "q4_attention.cu",
           "q4_attention_f16.cu", "q4_attention_bf16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


TORCH_SOURCE = "pkv_torch.cpp"


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")
    return path


def library_path() -> str:
    return os.path.join(LIB_DIR, "libpkv.so")


def torch_module_path() -> str:
    return os.path.join(LIB_DIR, "_pkv_torch.so")


def build_torch_module(out_path: str | None = None) -> str:
    """Compiles the extension module (CPython API, torch's tensor and CUDA stream headers)."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    out = out_path or torch_module_path()
    os.makedirs(os.path.dirname(out), exist_ok=True)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    lib = os.path.join(base, "lib")
    tmp = f"{out}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for i in includes for a in ("-isystem", i)], os.path.join(CSRC, TORCH_SOURCE), "-o", tmp,
           "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {TORCH_SOURCE}:\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(extra_flags=(), out_path: str | None = None, verbose_ptxas: bool = False) -> str:
    out = out_path or library_path()
    obj_dir = os.path.join(os.path.dirname(out), "obj")
    os.makedirs(obj_dir, exist_ok=True)
    flags = [*ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
             "-I", os.path.join(ROOT, "include"), *extra_flags]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [nvcc(), *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose_ptxas:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        module = ex.submit(build_torch_module, os.path.join(os.path.dirname(out), "_pkv_torch.so"))
        objs = list(ex.map(compile_one, SOURCES))
    tmp = f"{out}.{os.getpid()}.tmp"
    subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, out)
    # the library needs nothing of torch's headers: it is there even where the
    # module's compilation failed, which is reported now
    module.result()
    return out


if __name__ == "__main__":
    print(build(verbose_ptxas="--verbose-ptxas" in sys.argv))

"""Builds the CUDA library ``_lib/libmla_dcp.so`` for sm_103a and the Python
module ``_lib/_binding.so`` over it (in-tree).

Each translation unit is compiled in parallel with one ``-gencode`` and the
objects are linked into one shared library with the CUDA runtime linked
statically, so the library loads on a machine without a GPU driver (the
driver is looked up at first use).  The module is host code against PyTorch's
C++ headers; it finds the library beside itself.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libmla_dcp.so")
SOURCES = ["partial.cu", "partial_fp8.cu", "wuv_gemm.cu", "plan_merge.cu", "combine.cu", "capi.cu", "noalloc.cu", "gqa.cu",
           "gqa_fp8.cu", "append.cu"]
HEADERS = ["common.cuh", "merge.cuh", "ptx.cuh", "host_util.h", "rope.cuh"]
BINDING = os.path.join(OUT_DIR, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home():
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def nvcc():
    exe = os.path.join(_cuda_home(), "bin", "nvcc")
    return exe if os.path.exists(exe) else (shutil.which("nvcc") or "nvcc")


INCLUDE = os.path.join(os.path.dirname(HERE), "include")


def flags(extra=()):
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-I" + INCLUDE, *extra]


def _inputs():
    root = os.path.dirname(HERE)
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [BINDING_SOURCE] +
            [os.path.join(root, "include", "mla_dcp.h")])


def needs_build():
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(p) > t for p in _inputs())


def _binding_object(obj):
    """Compiles the Python module; returns what its link needs."""
    import torch
    home = os.path.dirname(torch.__file__)
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
           "-isystem", sysconfig.get_paths()["include"]]
    for d in (os.path.join(home, "include"),
              os.path.join(home, "include", "torch", "csrc", "api", "include"),
              os.path.join(_cuda_home(), "include")):
        cmd += ["-isystem", d]
    r = subprocess.run(cmd + [BINDING_SOURCE, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return os.path.join(home, "lib")


def build(force=False, verbose=False, extra_flags=()):
    if not (force or needs_build()):
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    objs = [os.path.join(OUT_DIR, os.path.splitext(s)[0] + ".o") for s in SOURCES]

    def compile_one(src, obj):
        cmd = [nvcc(), *flags(extra_flags), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return r.stdout + r.stderr

    binding_obj = os.path.join(OUT_DIR, "binding.o")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_lib = ex.submit(_binding_object, binding_obj)
        logs = list(ex.map(compile_one, SOURCES, objs))
        torch_lib = torch_lib.result()
    if verbose:
        for log in logs:
            if log.strip():
                print(log)
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", BINDING, binding_obj, "-L" + OUT_DIR,
           "-l:" + os.path.basename(LIB), "-L" + torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the Python module failed:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    import sys
    extra = ["-Xptxas", "-v"] if "-v" in sys.argv else []
    print(build(force=True, verbose=bool(extra), extra_flags=extra))

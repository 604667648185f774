"""Builds the CUDA library ``_lib/libmla_dcp.so`` for sm_103a and the Python
module ``_lib/_binding.so`` over it (in-tree).

Each translation unit is compiled in parallel with one ``-gencode`` and the
objects are linked into one shared library with the CUDA runtime linked
statically, so the library loads on a machine without a GPU driver (the
driver is looked up at first use).  The module is host code against PyTorch's
C++ headers; it finds the library beside itself.  The library is built and
loaded without it: what breaks the module's build takes only its own calls.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libmla_dcp.so")
SOURCES = ["partial.cu", "partial_fp8.cu", "wuv_gemm.cu", "plan_merge.cu", "combine.cu", "capi.cu", "noalloc.cu", "gqa.cu",
           "gqa_fp8.cu", "append.cu", "evict.cu", "weights.cu",
           "prefix.cu"]
HEADERS = ["common.cuh", "merge.cuh", "ptx.cuh", "host_util.h", "rope.cuh", "qterms.cuh",
           "pair.cuh", "prefix.h", "unit_merge.cuh"]
BINDING = os.path.join(OUT_DIR, "_binding.so")
BINDING_STAMP = os.path.join(OUT_DIR, "_binding.built-for")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home():
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def nvcc():
    exe = os.path.join(_cuda_home(), "bin", "nvcc")
    return exe if os.path.exists(exe) else (shutil.which("nvcc") or "nvcc")


INCLUDE = os.path.join(os.path.dirname(HERE), "include")
API_HEADER = os.path.join(INCLUDE, "mla_dcp.h")


def flags(extra=()):
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-I" + INCLUDE, *extra]


def _newer_than(t, paths):
    return any(os.path.getmtime(p) > t for p in paths)


def needs_build():
    """Whether the library is missing or older than one of its sources."""
    if not os.path.exists(LIB):
        return True
    return _newer_than(os.path.getmtime(LIB),
                       [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [API_HEADER])


def _binding_for():
    """What the Python module is compiled against besides its sources."""
    import torch
    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, python {sys.version}"


def needs_binding():
    """Whether the Python module is missing, older than one of its sources or
    compiled against another torch or Python."""
    if not (os.path.exists(BINDING) and os.path.exists(BINDING_STAMP)):
        return True
    with open(BINDING_STAMP) as f:
        if f.read() != _binding_for():
            return True
    return _newer_than(os.path.getmtime(BINDING), [BINDING_SOURCE, API_HEADER])


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

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        logs = list(ex.map(compile_one, SOURCES, objs))
    if verbose:
        for log in logs:
            if log.strip():
                print(log)
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return LIB


def build_binding(force=False):
    """Builds the Python module, and the library if that is not up to date."""
    if not (force or needs_binding()):
        build()
        return BINDING
    os.makedirs(OUT_DIR, exist_ok=True)
    obj = os.path.join(OUT_DIR, "binding.o")
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        torch_lib = ex.submit(_binding_object, obj)
        build(force)
        torch_lib = torch_lib.result()
    if os.path.exists(BINDING_STAMP):
        os.remove(BINDING_STAMP)
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", BINDING, obj, "-L" + OUT_DIR,
           "-l:" + os.path.basename(LIB), "-L" + torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the Python module failed:\n{r.stdout}\n{r.stderr}")
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_for())
    return BINDING


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "-v" in sys.argv else []
    print(build(force=True, verbose=bool(extra), extra_flags=extra))
    print(build_binding())

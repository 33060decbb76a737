"""In-tree build of the CUDA library libw4a16.so for sm_103a, and of the
binding's small host extension.

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library next to this file (``_lib/libw4a16.so``) with the CUDA runtime
linked statically.  Used by ``__graft_entry__.build()``."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libw4a16.so")
MARSHAL = os.path.join(OUT_DIR, "_marshal.so")  # the binding's host extension (csrc/marshal.cpp)
SOURCES = ["api.cu", "dequant.cu", "gemv_int4.cu", "gemv_chain.cu", "moe_fp4.cu", "moe_fp4_gemm.cu",
           "gemm_int4_tc.cu", "gemm_int4_f16.cu", "gemm_bf16_tc.cu", "copy.cu",
           "api_kv4.cu", "kv4_plan.cu", "kv4_rope.cu", "kv4_attention.cu", "kv4_prompt.cu", "kv4_sparse.cu", "kv4_prefix.cu",
           "kv4_select.cu", "sample.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def build_marshal() -> str:
    """The host extension that checks tensors and makes calls for the binding."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), INCLUDE,
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = MARSHAL + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), *["-I" + d for d in inc],
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for marshal.cpp:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, MARSHAL)
    return MARSHAL


def _stale(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile what is older than any source or header, the library and the
    host extension; return the library's path.  The library does not need the
    extension: it is in place where compiling that one fails (which raises)."""
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "w4a16.h"))
    deps.append(os.path.abspath(__file__))
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = ex.submit(build_marshal) if force or _stale(MARSHAL, deps) else None
        if force or _stale(LIB, deps):
            build_library(verbose, extra_flags)
        if marshal:
            marshal.result()
    return LIB


def build_library(verbose: bool = False, extra_flags=()) -> None:
    """Compile and link libw4a16.so."""
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [nvcc()] + NVCC_FLAGS + list(extra_flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True))

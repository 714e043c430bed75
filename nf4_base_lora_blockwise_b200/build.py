"""Build libqlora_nf4.so in-tree with nvcc for sm_100a, and the torch binding over it.

    python -m nf4_base_lora_blockwise_b200.build [-v]

Each ``csrc/*.cu`` is compiled to an object under ``_build/`` (in parallel), then linked into
``nf4_base_lora_blockwise_b200/libqlora_nf4.so`` next to this file.  Objects are rebuilt when
their source or any header is newer.  Only the C ABI (``include/qlora_nf4.h``) is exported.
``csrc/torch_bind.cpp``, the CPython extension of ``block`` and ``optim``, is compiled with the host
compiler against torch's headers into ``_torch_bind.so`` beside the library.
"""

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqlora_nf4.so")
BIND = os.path.join(PKG, "_torch_bind.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
         "-fvisibility=hidden", "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_commands():
    """(compile, link) of the torch binding: torch's include paths and libraries, the interpreter's
    headers, and libqlora_nf4.so found beside it."""
    import torch
    from torch.utils import cpp_extension
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    obj = os.path.join(BUILD, "torch_bind.cpp.o")
    src = os.path.join(CSRC, "torch_bind.cpp")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], cuda]
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *("-isystem" + p for p in inc), "-c", src, "-o", obj]
    # The shared C++ runtime, whatever the compiler's default: exceptions and streams cross into torch,
    # which has its own copy of a static one otherwise.
    link = [cxx, "-shared", "-nostdlib++", obj, "-o", BIND, "-L" + PKG, "-l:libqlora_nf4.so",
            "-Wl,-rpath,$ORIGIN", *("-L" + p for p in cpp_extension.library_paths()),
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-l:libstdc++.so.6"]
    return src, obj, compile_, link


def build(verbose=False, ptxas_verbose=False):
    """Compile and link the library; returns its path.  Raises on any compiler error."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if ptxas_verbose or _stale(obj, [src] + hdrs):
            cmd = [nvcc] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + [
                "-c", src, "-o", obj]
            jobs.append(cmd)

    bind_src, bind_obj, bind_compile, bind_link = _bind_commands()
    if _stale(bind_obj, [bind_src, os.path.join(ROOT, "include", "qlora_nf4.h")]):
        jobs.insert(0, bind_compile)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        p = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, p

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, os.cpu_count() or 1)) as ex:
        for cmd, p in ex.map(run, jobs):
            if verbose or ptxas_verbose:
                sys.stdout.write(p.stdout)
                sys.stderr.write(p.stderr)
            if p.returncode != 0:
                raise RuntimeError("compiler failed:\n" + " ".join(cmd) + "\n" + p.stdout + p.stderr)
    if jobs or _stale(LIB, objs):
        cmd = [nvcc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", LIB] + objs + [
            "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + p.stdout + p.stderr)
    if _stale(BIND, [bind_obj]):
        cmd, p = run(bind_link)
        if p.returncode != 0:
            raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + p.stdout + p.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)

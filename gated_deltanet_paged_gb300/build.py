"""Build the CUDA library libgdn_paged.so in-tree (nvcc, sm_103a only), and the
Python binding of its attention calls, _attention.so.

Each csrc/*.cu compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so loading it needs no
driver (symbols can be inspected on a machine without a GPU).  csrc/binding.cpp
compiles beside them against torch's headers and links to the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgdn_paged.so")
BINDING = os.path.join(HERE, "_attention.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".cpp"))]
    files.append(os.path.join(INCLUDE, "gdn_paged.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _deps())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))


def _torch_paths():
    """(include flags, library folder) of the installed torch."""
    import torch

    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"),
               sysconfig.get_paths()["include"], INCLUDE]
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi())
    return [abi] + ["-I" + p for p in include], os.path.join(root, "lib")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc/, link libgdn_paged.so and _attention.so; returns the library's path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE,
                    "--expt-relaxed-constexpr"] + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    torch_flags, torch_lib = _torch_paths()

    def compile_binding():
        obj = os.path.join(BUILD, "binding.o")
        _run(["g++", "-O2", "-std=c++17", "-fPIC"] + torch_flags + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj],
             "g++ on binding.cpp")
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, srcs))
        binding = binding.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    _run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs, "link")
    os.replace(tmp, LIB)
    tmp = BINDING + ".%d.tmp" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, binding, "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-L" + HERE, "-l:libgdn_paged.so", "-Wl,-rpath,$ORIGIN"], "link of the binding")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    extra = sys.argv[1:]
    print(build(force=True, verbose=True, extra_flags=extra))

"""Build the CUDA library libgdn_paged.so in-tree (nvcc, sm_103a only), and the
Python binding of its attention calls, _attention.so.

Each csrc/*.cu compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so loading it needs no
driver (symbols can be inspected on a machine without a GPU).  csrc/binding.cpp
compiles against torch's headers and links to the library; neither the library
nor the recurrent layer's calls need it.
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
HEADER = os.path.join(INCLUDE, "gdn_paged.h")
BINDING = os.path.join(HERE, "_attention.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_KEY = os.path.join(BUILD, "binding.txt")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(target, files):
    """Whether `target` is there and no older than any of the files."""
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def up_to_date() -> bool:
    """The library."""
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    return _newer(LIB, sources() + headers + [HEADER])


def _binding_key() -> str:
    """What the binding was compiled against."""
    import torch

    return "%s %s %s" % (sysconfig.get_config_var("SOABI"), torch.__version__, os.path.dirname(torch.__file__))


def binding_up_to_date() -> bool:
    """The binding, and that it was built for this Python and this torch."""
    if not _newer(BINDING, [BINDING_SRC, HEADER]) or not os.path.exists(BINDING_KEY):
        return False
    with open(BINDING_KEY, encoding="utf-8") as f:
        return f.read() == _binding_key()


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


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc/*.cu and link libgdn_paged.so; needs nvcc alone.  Returns its path."""
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

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".%d.tmp" % os.getpid()
    _run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs, "link")
    os.replace(tmp, LIB)
    return LIB


def _compile_binding():
    """binding.o, and torch's library folder."""
    os.makedirs(BUILD, exist_ok=True)
    flags, torch_lib = _torch_paths()
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC"] + flags + ["-c", BINDING_SRC, "-o", obj], "g++ on binding.cpp")
    return obj, torch_lib


def _link_binding(obj, torch_lib):
    tmp = BINDING + ".%d.tmp" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-L" + HERE, "-l:libgdn_paged.so", "-Wl,-rpath,$ORIGIN"], "link of the binding")
    if os.path.exists(BINDING_KEY):
        os.remove(BINDING_KEY)  # no moment at which an old key stands beside a new binding
    os.replace(tmp, BINDING)
    with open(BINDING_KEY + ".%d.tmp" % os.getpid(), "w", encoding="utf-8") as f:
        f.write(_binding_key())
    os.replace(f.name, BINDING_KEY)


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp against the installed torch and link _attention.so
    to the library, which is there already; returns its path."""
    if force or not binding_up_to_date():
        _link_binding(*_compile_binding())
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Both, side by side; returns the library's path.  The library is in place
    even where the binding cannot be built."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding) if force or not binding_up_to_date() else None
        build_library(force, verbose, extra_flags)
        if binding:
            _link_binding(*binding.result())
    return LIB


if __name__ == "__main__":
    extra = sys.argv[1:]
    print(build(force=True, verbose=True, extra_flags=extra))

"""Build libarfusion.so in-tree with nvcc for sm_103a (no cmake).

Each translation unit compiles in parallel; the shared library links the
CUDA runtime dynamically so it shares one runtime with PyTorch.  Beside it
``_marshal.<PyTorch and Python>.so``, the binding's argument marshalling against
PyTorch's headers.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libarfusion.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def marshal_path() -> str:
    """Where the marshalling module for this PyTorch and this Python lies.  It reads
    tensors through PyTorch's inlined code: one built for another version may load,
    its symbols resolved, and read the wrong bytes, so its name says which it is for."""
    import torch
    tag = (f"{torch.__version__}-{(torch.version.git_version or 'none')[:12]}"
           f"-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}-{sysconfig.get_config_var('SOABI')}")
    return os.path.join(HERE, f"_marshal.{tag}.so")


def marshal_command(out: str) -> list[str]:
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    include = os.path.join(root, "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", include,
            "-I", os.path.join(include, "torch", "csrc", "api", "include"),
            "-I", os.path.join(os.path.dirname(cuda_lib_dir()), "include"),
            "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.cpp"), "-o", out,
            "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            f"-Wl,-rpath,{lib}"]


def build_marshal(path: str) -> None:
    """marshal.cpp against the installed PyTorch.  The binding works without it,
    through ctypes: a failure is told and noted beside `path`, and not tried again
    until a source changes."""
    tmp = path + f".tmp{os.getpid()}"
    try:
        r = subprocess.run(marshal_command(tmp), capture_output=True, text=True)
        why = r.stderr if r.returncode else None
    except OSError as e:                        # no compiler
        why = str(e)
    if why is None:
        os.replace(tmp, path)
        return
    if os.path.exists(path):                    # an older one must not stay
        os.remove(path)
    with open(path + ".failed", "w") as f:
        f.write(why)
    sys.stderr.write(f"marshal.cpp not built (calls go through ctypes):\n{why}\n")


def fresh(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= deps_mtime()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    try:
        path = marshal_path()
    except ImportError as e:                    # no PyTorch: the library alone
        sys.stderr.write(f"marshal.cpp not built: {e}\n")
        return build_library(force, verbose, extra_flags)
    if force or not (fresh(path) or fresh(path + ".failed")):
        with ThreadPoolExecutor(1) as ex:
            marshal = ex.submit(build_marshal, path)
            build_library(force, verbose, extra_flags)
            marshal.result()
        return LIB
    return build_library(force, verbose, extra_flags)


def build_library(force: bool, verbose: bool, extra_flags) -> str:
    if not force and fresh(LIB):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nv = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nv, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nv, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", f"-rpath,{cuda_lib_dir()}",
           *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

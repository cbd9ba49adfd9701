"""Build libadafuse.so in-tree with nvcc for sm_100a (no GPU needed; neither
torch nor Python's headers), and the Python binding of the operators with the
host compiler, for the Python and the torch that run this."""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libadafuse.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-shared", "-cudart", "static",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(CSRC, "*.h")))
            + [os.path.join(os.path.dirname(HERE), "include", "adafuse.h")])


def newer_than(target: str, files) -> bool:
    """Whether `target` exists and none of the files was changed after it."""
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def up_to_date() -> bool:
    return newer_than(LIB, sources() + headers())


def binding_path() -> str:
    """The binding's file, named after what its object code is tied to: Python's
    and torch's binary interfaces.  After either was replaced it is another
    file, which is built or found missing, but never the old one loaded."""
    import sysconfig

    import torch
    return os.path.join(HERE, f"_binding.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}"
                              f"-{(torch.version.git_version or '')[:8]}.so")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    source = os.path.join(CSRC, "binding.cpp")
    inc = os.path.join(os.path.dirname(HERE), "include")
    target = binding_path()
    if not force and newer_than(target, [source, os.path.join(inc, "adafuse.h")]):
        return target
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    others = [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
              os.path.join(root, "include")]
    tmp = target + f".tmp{os.getpid()}"
    # the system's compiler, whose C++ runtime is the one that torch's libraries
    # load: one that links a runtime of its own cannot catch their exceptions
    gxx = "/usr/bin/g++" if os.path.exists("/usr/bin/g++") else "g++"
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wextra",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", inc,
           *(f for d in others for f in ("-isystem", d)), source, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, target)
    return target


def build_library(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    inc = os.path.join(os.path.dirname(HERE), "include")
    cmd = [NVCC, *FLAGS, "-I", inc, *extra, "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The library first, which needs nvcc alone; then, where there is a torch
    to bind it to, the operators' binding."""
    build_library(force, verbose, extra)
    if importlib.util.find_spec("torch") is not None:
        build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    import sys
    build(force=True, verbose=True, extra=sys.argv[1:])
    print(LIB)
